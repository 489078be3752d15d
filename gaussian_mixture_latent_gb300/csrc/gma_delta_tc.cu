// The gated delta rule in chunks of 64 rows on the tensor cores (bf16 inputs, d <= 128, d and dv multiples of 8).
//
// Within a chunk, with G the running sum of the log decays, D_ij = e^{G_i - G_j} (i >= j), L_ij = D_ij k_i.k_j below
// the diagonal and S the state [d, dv] before the chunk:
//   W = (I + L diag(beta))^-1 (V - diag(e^G) K S),   U = diag(beta) W
//   O = scale (diag(e^G) Q S + (D o Q K^T) U),       S <- e^{G_C} S + (diag(e^{G_C - G}) K)^T U.
// Every exponent is a difference that is <= 0 for decays <= 0; G is summed in fp64 and kept as two floats, so that
// differences of large sums are exact to fp32.
//
// The state never leaves registers.  A chain warp holds S^T for 16 columns of dv, [16, d] as fp32 accumulator tiles.
// Written transposed, every product of the chain has such a tile on its left:
//   (K S)^T = S^T K^T,  W^T = R^T T^T,  O^T = S^T Q^T + U^T P^T,  S^T += (f U)^T K,
// and an accumulator tile is the next product's A operand as it stands: no exchange between threads.  The right sides
// (K, Q, and T = (I + L diag(beta))^-1, P = scale D o Q K^T) are read from shared memory with ldmatrix.
//
// Four prep warps of the same CTA make T and P of chunk c + 1 while the chain warps take chunk c, and load chunk c + 2.
// T is inverted in fp32: 16 x 16 diagonal blocks by substitution (a product of powers would overflow for repeated
// keys), joined to 32 and 64 by X21 = -T22 (A21 T11) with three-term products.
//
// Precision.  K, Q, V are bf16 as given and exact.  fp32 values that enter a product (S, R, U, T) are split into
// NT bf16 terms: three (24 bits) when the state is returned, two (16 bits, 2^-17) when only the bf16 output is;
// P has two.  The output's own products take S and U in one term: 2^-9 at most of the result's scale, below the
// output's rounding of 2^-8... each counted in the tests' tolerance.
//
// Bound by the chain's mma.sync issue: measured 8.0 cycles for an m16n8k16 on each of the SM's four tensor units
// (1024 multiply-adds a cycle and SM, whatever the number of warps), latency 21.  tcgen05 is four times that rate but
// has its accumulators in TMEM: the three dependent products of a chunk would each pay a round trip through registers
// and shared memory (load, convert, store, fence) of the same order as this whole step.
#include <cstdint>

#include "gma_delta.h"
#include "gma_delta_mma.cuh"

namespace gma {
namespace {

using namespace dmma;

constexpr int C = kTcRows, kStages = 3, kVec = 3;
constexpr int kChain = 128, kPrep = 256, kThreads = kChain + kPrep;
// Registers: the block is launched with 168 a thread (384 x 168 = 64512); the chain's warpgroup takes 240 and the two
// prep warpgroups keep 128 (128 x 240 + 256 x 128 = 63488).
constexpr int kChainRegs = 240, kPrepRegs = 128;
enum { kBarPrep = 1, kBarAll = 2, kBarInv = 3, kBarPair = 4 };       // named barriers; pairs use 4..7

struct TcArgs {
    DeltaProblem p;
    const float *state_in;
    float *state_out;
    void *out;
    int groups;                        // CTAs of one head
};

struct Vec {                           // one chunk's row factors
    float2 G[C];                       // running sum of the log2 decays, hi + lo
    float e[C], f[C], beta[C];         // e^G, e^{G_C - G}
    float last, pad[3];                // e^{G_C}
};

template <int D, int NT, int SL>
struct Smem {
    static constexpr int kRow = 2 * D, kKey = C * kRow, kValRow = 32 * SL, kVal = C * kValRow;
    static constexpr int kT = NT * kTriBytes, kP = 2 * kTriBytes;
    static constexpr int oK = 0, oQ = oK + kStages * kKey, oV = oQ + kStages * kKey, oT = oV + kStages * kVal;
    static constexpr int oP = oT + 2 * kT, oA = oP + 2 * kP, oI = oA + C * kFp * 4, oX = oI + C * kFp * 4;
    static constexpr int oVec = oX + 4 * 32 * 12 * 4, total = oVec + kVec * (int)sizeof(Vec);
};

template <int D, int NT, int SL>
__global__ void __launch_bounds__(kThreads, 1) delta_tc_kernel(const TcArgs a) {
    using L = Smem<D, NT, SL>;
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

    {   // rows that do not exist
        const int w = min(16 * SL, p.dv - c0);
        for (size_t i = tid; i < (size_t)(p.N - len) * (w / 8); i += blockDim.x) {
            const size_t r = len + i / (w / 8);
            *reinterpret_cast<uint4 *>(out + (vrow + r) * p.dv + c0 + (int)(i % (w / 8)) * 8) = make_uint4(0, 0, 0, 0);
        }
    }

    constexpr int kSync = 32 * SL + kPrep;               // threads of the barrier between chunks
    if (tid >= kChain) {
        // ------------------------------------------------------------------------------------------ prep warps
        asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kPrepRegs));
        const int pt = tid - kChain, pw = (pt >> 5) & 3;
        const bool inv = pt < 128;                       // warps 0-3: K K^T and the inverse; 4-7: Q K^T, loads, decays
        const __nv_bfloat16 *K = static_cast<const __nv_bfloat16 *>(p.Kx), *Q = static_cast<const __nv_bfloat16 *>(p.Qx);
        const __nv_bfloat16 *V = static_cast<const __nv_bfloat16 *>(p.V);
        auto load = [&](int c) {
            if (c < nc) {
                const int st = c % kStages, lt = pt - 128;
                for (int i = lt; i < C * (D / 8); i += 128) {
                    const int r = i / (D / 8), col = i % (D / 8), row = c * C + r;
                    const bool ok = row < len && col * 8 < p.d;
                    const size_t off = ok ? (krow + row) * p.d + col * 8 : 0;
                    copy16(sb + L::oK + st * L::kKey + at<L::kRow>(r, col), K + off, ok);
                    copy16(sb + L::oQ + st * L::kKey + at<L::kRow>(r, col), Q + off, ok);
                }
                for (int i = lt; i < C * 2 * SL; i += 128) {
                    const int r = i / (2 * SL), col = i % (2 * SL), row = c * C + r;
                    const bool ok = row < len && c0 + col * 8 < p.dv;
                    const size_t off = ok ? (vrow + row) * p.dv + c0 + col * 8 : 0;
                    copy16(sb + L::oV + st * L::kVal + at<L::kValRow>(r, col), V + off, ok);
                }
            }
            copy_commit();
        };
        // the decays, by one warp (the one with the least of Q K^T): read a chunk ahead, two rows to a lane
        float gn[2] = {0.f, 0.f}, bn[2] = {0.f, 0.f};
        auto read_gates = [&](int c) {
#pragma unroll
            for (int j = 0; j < 2; ++j) {
                const int row = c * C + 2 * lane + j;
                gn[j] = bn[j] = 0.f;
                if (row < len) {
                    gn[j] = delta_floor(delta_gate(p.g, vrow + row, p.gate_bf16));
                    bn[j] = delta_gate(p.beta, vrow + row, p.gate_bf16);
                }
            }
        };
        auto decays = [&](int c) {
            Vec &vec = reinterpret_cast<Vec *>(sm + L::oVec)[c % kVec];
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
        };
        float *A = reinterpret_cast<float *>(sm + L::oA), *I = reinterpret_cast<float *>(sm + L::oI);
        float *X = reinterpret_cast<float *>(sm + L::oX) + pw * 32 * 12;
        const int r0 = lane >> 2, q0 = 2 * (lane & 3);

        auto prep = [&](int c) {
            const int st = c % kStages, bf = c & 1;
            const Vec &vec = reinterpret_cast<const Vec *>(sm + L::oVec)[c % kVec];
            const uint32_t kt = sb + L::oK + st * L::kKey, xt = inv ? kt : sb + L::oQ + st * L::kKey;
            const int ar = (lane & 7) + ((lane >> 3) & 1) * 8, ac = lane >> 4;      // A operand: row, 16-byte piece
            const int br = (lane & 7) + (lane >> 4) * 8, bc = (lane >> 3) & 1;      // B operand of two n tiles
            // rows 16 pw.. of K K^T (Q K^T), up to the diagonal
            float x[8][4];
#pragma unroll
            for (int n = 0; n < 8; ++n)
#pragma unroll
                for (int j = 0; j < 4; ++j) x[n][j] = 0.f;
#pragma unroll
            for (int ks = 0; ks < D / 16; ++ks) {
                uint32_t fa[4];
                ldsm(fa, xt + at<L::kRow>(pw * 16 + ar, 2 * ks + ac));
#pragma unroll
                for (int np = 0; np < 4; ++np) {
                    if (np > pw) continue;
                    uint32_t fb[4];
                    ldsm(fb, kt + at<L::kRow>(np * 16 + br, 2 * ks + bc));
                    mma(x[2 * np], fa, fb[0], fb[1]);
                    mma(x[2 * np + 1], fa, fb[2], fb[3]);
                }
            }
            char *P = sm + L::oP + bf * L::kP;
            const int i0 = pw * 16 + r0, i1 = i0 + 8;
            const float2 g0 = vec.G[i0], g1 = vec.G[i1];
#pragma unroll
            for (int n = 0; n < 8; ++n) {
                if (n / 2 > pw) continue;
                const int j = 8 * n + q0;
                const float4 gj = *reinterpret_cast<const float4 *>(vec.G + j);      // hi, lo of rows j and j + 1
                float m0, m1;                            // the columns' factors: beta, or the output's scale
                if (inv) {
                    const float2 be = *reinterpret_cast<const float2 *>(vec.beta + j);
                    m0 = be.x; m1 = be.y;
                } else {
                    m0 = m1 = p.scale;
                }
                x[n][0] *= ex2((g0.x - gj.x) + (g0.y - gj.y)) * m0;
                x[n][1] *= ex2((g0.x - gj.z) + (g0.y - gj.w)) * m1;
                x[n][2] *= ex2((g1.x - gj.x) + (g1.y - gj.y)) * m0;
                x[n][3] *= ex2((g1.x - gj.z) + (g1.y - gj.w)) * m1;
                if (n / 2 == pw) {                       // the diagonal block: below (and, for P, on) the diagonal
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
                    const uint32_t o = tri(pw, n / 2) + 4 * (lane & 3);
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
            } else if (pw == 0) {
                decays(c + 1);
                read_gates(c + 2);
            }
            bar<kPrep>(kBarPrep);
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
            bar<kPrep>(kBarPrep);
            char *T = sm + L::oT + bf * L::kT;
#pragma unroll
            for (int u = 0; u < 10 * 128 / kPrep; ++u) { // pairs of the ten blocks
                const int e = pt + u * kPrep, blk = e >> 7, r = (e >> 3) & 15, pc = e & 7;
                const int ib = blk >= 6 ? 3 : blk >= 3 ? 2 : blk >= 1 ? 1 : 0, jb = blk - ib * (ib + 1) / 2;
                const float2 y = *reinterpret_cast<const float2 *>(I + (16 * ib + r) * kFp + 16 * jb + 2 * pc);
                uint32_t t[NT];
                split<NT>(y.x, y.y, t);
#pragma unroll
                for (int k = 0; k < NT; ++k)
                    *reinterpret_cast<uint32_t *>(T + k * kTriBytes + blk * 512 + at<32>(r, pc >> 2) + 4 * (pc & 3)) = t[k];
            }
        };

        if (!inv) {
            load(0);
            load(1);
            if (pw == 0) {
                read_gates(0);
                decays(0);
                read_gates(1);
            }
            copy_wait<1>();
        }
        bar<kPrep>(kBarPrep);
        if (nc > 0) prep(0);
        bar<kSync>(kBarAll);
        for (int c = 0; c < nc; ++c) {
            if (!inv) {
                load(c + 2);
                copy_wait<1>();
            }
            bar<kPrep>(kBarPrep);                        // chunk c + 1 is there; T's fp32 form has been read
            if (c + 1 < nc) prep(c + 1);
            bar<kSync>(kBarAll);
        }
        if (!inv) copy_wait<0>();
        return;
    }
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kChainRegs));
    if (warp >= SL) return;

    // ---------------------------------------------------------------------------------------------- chain warps
    const int col = c0 + 16 * warp + (lane >> 2), q0 = 2 * (lane & 3);
    const size_t sbase = (size_t)bh * p.d * p.dv;
    float S[D / 8][4];                                   // S^T: rows col, col + 8; columns 8 n + q0, + 1
#pragma unroll
    for (int n = 0; n < D / 8; ++n)
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const int r = 8 * n + q0 + (j & 1), c = col + 8 * (j >> 1);
            S[n][j] = a.state_in && r < p.d && c < p.dv ? a.state_in[sbase + (size_t)r * p.dv + c] : 0.f;
        }
    const int br = (lane & 7) + (lane >> 4) * 8, bc = (lane >> 3) & 1;              // B operand: rows n, pieces k
    const int tr = (lane & 7) + ((lane >> 3) & 1) * 8, tc = lane >> 4;              // transposed: rows k, pieces n
    bar<kSync>(kBarAll);
    for (int c = 0; c < nc; ++c) {
        const int st = c % kStages, bf = c & 1;
        const uint32_t kt = sb + L::oK + st * L::kKey, qt = sb + L::oQ + st * L::kKey, vt = sb + L::oV + st * L::kVal;
        const uint32_t tt = sb + L::oT + bf * L::kT, pt = sb + L::oP + bf * L::kP;
        const Vec &vec = reinterpret_cast<const Vec *>(sm + L::oVec)[c % kVec];
        float y[8][4], o[8][4];
#pragma unroll
        for (int n = 0; n < 8; ++n)
#pragma unroll
            for (int j = 0; j < 4; ++j) y[n][j] = o[n][j] = 0.f;
        // y = (K S)^T in NT terms of S, o = (Q S)^T in one
#pragma unroll
        for (int ks = 0; ks < D / 16; ++ks) {
            uint32_t fs[NT][4];
            split_a<NT>(S[2 * ks], S[2 * ks + 1], fs);
#pragma unroll
            for (int np = 0; np < 4; ++np) {
                uint32_t fb[4], fq[4];
                ldsm(fb, kt + at<L::kRow>(np * 16 + br, 2 * ks + bc));
                ldsm(fq, qt + at<L::kRow>(np * 16 + br, 2 * ks + bc));
#pragma unroll
                for (int t = NT - 1; t >= 0; --t) {
                    mma(y[2 * np], fs[t], fb[0], fb[1]);
                    mma(y[2 * np + 1], fs[t], fb[2], fb[3]);
                }
                mma(o[2 * np], fs[0], fq[0], fq[1]);
                mma(o[2 * np + 1], fs[0], fq[2], fq[3]);
            }
        }
        // R = V - e^G K S, the left operand of T
        uint32_t fr[4][NT][4];
#pragma unroll
        for (int np = 0; np < 4; ++np) {
            uint32_t fv[4];
            ldsm_t(fv, vt + at<L::kValRow>(np * 16 + br, 2 * warp + bc));
#pragma unroll
            for (int m = 0; m < 2; ++m) {
                const int n = 2 * np + m;
                const float2 e = *reinterpret_cast<const float2 *>(vec.e + 8 * n + q0);
                y[n][0] = fmaf(-e.x, y[n][0], low(fv[2 * m]));
                y[n][1] = fmaf(-e.y, y[n][1], high(fv[2 * m]));
                y[n][2] = fmaf(-e.x, y[n][2], low(fv[2 * m + 1]));
                y[n][3] = fmaf(-e.y, y[n][3], high(fv[2 * m + 1]));
#pragma unroll
                for (int j = 0; j < 4; ++j) o[n][j] *= p.scale * ((j & 1) ? e.y : e.x);
            }
            split_a<NT>(y[2 * np], y[2 * np + 1], fr[np]);
        }
        // W^T = R^T T^T over the blocks at and below the diagonal
#pragma unroll
        for (int n = 0; n < 8; ++n)
#pragma unroll
            for (int j = 0; j < 4; ++j) y[n][j] = 0.f;
#pragma unroll
        for (int ib = 0; ib < 4; ++ib)
#pragma unroll
            for (int jb = 0; jb <= ib; ++jb) {
#pragma unroll
                for (int t = NT - 1; t >= 0; --t) {
                    uint32_t fb[4];
                    ldsm(fb, tt + t * kTriBytes + tri(ib, jb) + at<32>(br, bc));
#pragma unroll
                    for (int s = NT - 1 - t; s >= 0; --s) {
                        mma(y[2 * ib], fr[jb][s], fb[0], fb[1]);
                        mma(y[2 * ib + 1], fr[jb][s], fb[2], fb[3]);
                    }
                }
            }
        // U = beta W; O += U P^T (two terms each)
        uint32_t fu[4][2][4];
#pragma unroll
        for (int n = 0; n < 8; ++n) {
            const float2 be = *reinterpret_cast<const float2 *>(vec.beta + 8 * n + q0);
#pragma unroll
            for (int j = 0; j < 4; ++j) y[n][j] *= (j & 1) ? be.y : be.x;
        }
#pragma unroll
        for (int kb = 0; kb < 4; ++kb) split_a<2>(y[2 * kb], y[2 * kb + 1], fu[kb]);
#pragma unroll
        for (int ib = 0; ib < 4; ++ib)
#pragma unroll
            for (int jb = 0; jb <= ib; ++jb)
#pragma unroll
                for (int t = 1; t >= 0; --t) {
                    uint32_t fb[4];
                    ldsm(fb, pt + t * kTriBytes + tri(ib, jb) + at<32>(br, bc));
#pragma unroll
                    for (int s = 1 - t; s >= 0; --s) {
                        mma(o[2 * ib], fu[jb][s], fb[0], fb[1]);
                        mma(o[2 * ib + 1], fu[jb][s], fb[2], fb[3]);
                    }
                }
        // S <- e^{G_C} S + (f U)^T K
        const float last = vec.last;
#pragma unroll
        for (int n = 0; n < D / 8; ++n)
#pragma unroll
            for (int j = 0; j < 4; ++j) S[n][j] *= last;
#pragma unroll
        for (int kb = 0; kb < 4; ++kb) {
#pragma unroll
            for (int m = 0; m < 2; ++m) {
                const float2 f = *reinterpret_cast<const float2 *>(vec.f + 16 * kb + 8 * m + q0);
#pragma unroll
                for (int j = 0; j < 4; ++j) y[2 * kb + m][j] *= (j & 1) ? f.y : f.x;
            }
            uint32_t fs[NT][4];
            split_a<NT>(y[2 * kb], y[2 * kb + 1], fs);
#pragma unroll
            for (int nd = 0; nd < D / 16; ++nd) {
                uint32_t fb[4];
                ldsm_t(fb, kt + at<L::kRow>(kb * 16 + tr, 2 * nd + tc));
#pragma unroll
                for (int t = NT - 1; t >= 0; --t) {
                    mma(S[2 * nd], fs[t], fb[0], fb[1]);
                    mma(S[2 * nd + 1], fs[t], fb[2], fb[3]);
                }
            }
        }
        // O through the chunk's own V columns to memory
#pragma unroll
        for (int np = 0; np < 4; ++np)
            stsm_t(vt + at<L::kValRow>(np * 16 + br, 2 * warp + bc), pack(o[2 * np][0], o[2 * np][1]),
                   pack(o[2 * np][2], o[2 * np][3]), pack(o[2 * np + 1][0], o[2 * np + 1][1]),
                   pack(o[2 * np + 1][2], o[2 * np + 1][3]));
        __syncwarp();
        const int oc = c0 + 16 * warp + (lane & 1) * 8;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int r = i * 16 + (lane >> 1), row = c * C + r;
            if (row < len && oc < p.dv)
                *reinterpret_cast<uint4 *>(out + (vrow + row) * p.dv + oc) =
                    *reinterpret_cast<const uint4 *>(sm + L::oV + st * L::kVal + at<L::kValRow>(r, 2 * warp + (lane & 1)));
        }
        bar<kSync>(kBarAll);
    }
    if (a.state_out)
#pragma unroll
        for (int n = 0; n < D / 8; ++n)
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const int r = 8 * n + q0 + (j & 1), c = col + 8 * (j >> 1);
                if (r < p.d && c < p.dv) a.state_out[sbase + (size_t)r * p.dv + c] = S[n][j];
            }
}

template <int D, int NT, int SL>
cudaError_t launch(const TcArgs &args, cudaStream_t s) {
    TcArgs a = args;
    a.groups = (a.p.dv + 16 * SL - 1) / (16 * SL);
    const int smem = Smem<D, NT, SL>::total;
    static_assert(Smem<D, NT, SL>::total <= 227 * 1024, "shared memory");
    const cudaError_t e = set_dyn_smem((const void *)delta_tc_kernel<D, NT, SL>, smem);
    if (e != cudaSuccess) return e;
    delta_tc_kernel<D, NT, SL><<<(unsigned)(a.p.B * a.p.H * a.groups), kThreads, smem, s>>>(a);
    return cudaGetLastError();
}

template <int D, int NT>
cudaError_t by_slices(const TcArgs &a, cudaStream_t s) {
    // As few columns to a CTA as one wave of CTAs allows: the chain's time does not depend on the number of chain
    // warps (up to one to a tensor unit), and spreading them over SMs shares shared memory and prep among fewer.
    const long long heads = (long long)a.p.B * a.p.H, slices = (a.p.dv + 15) / 16;
    if (heads * slices <= 152) return launch<D, NT, 1>(a, s);
    if (heads * ((slices + 1) / 2) <= 152) return launch<D, NT, 2>(a, s);
    return launch<D, NT, 4>(a, s);
}

}  // namespace

bool delta_tc_supported(const DeltaProblem &p) {
    return p.bf16 && p.d <= 128 && p.d % 8 == 0 && p.dv % 8 == 0;
}

cudaError_t delta_tc_forward(const DeltaProblem &p, const float *state_in, void *out, float *state_out,
                             cudaStream_t s) {
    const TcArgs a{p, state_in, state_out, out, 0};
    if (p.d <= 64) return state_out ? by_slices<64, 3>(a, s) : by_slices<64, 2>(a, s);
    return state_out ? by_slices<128, 3>(a, s) : by_slices<128, 2>(a, s);
}

}  // namespace gma
