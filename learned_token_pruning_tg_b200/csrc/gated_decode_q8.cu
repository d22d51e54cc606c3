// gated_decode_q8.cu -- decoding steps of token-gated attention over an 8-bit KV cache.
//
// With codes K, V and one scale per block of 32 keys and head, for the R = n_q G query
// rows that read one KV head:
//   x_rc = (tau / sqrt(d)) kscale (q_r . K_c) + g_r s_c
//   out_r = sum_blocks vscale sum_{c in block} e^(x_rc - m_r) V_c / sum_c e^(x_rc - m_r)
// (in natural units, so that a bias of fp32's lowest number, a common mask, stays a number; a weight is
// 2^((x - m) log2 e), one multiplication more.)
// The cache is read once: 2 d bytes a key and head, so HBM bounds a long step and latency a
// short one.
//
// Work: a unit is one block (32 keys) of one head of one sequence.  Short caches give every head a thread block, or a
// cluster of up to 16 of them that merge their sums through distributed shared memory.  Else the units of all
// sequences, in order (sequence, head, block), are cut into equal runs, one for every SM (counted on the device from
// `lengths`, so one captured launch serves growing and ragged sequences evenly), and each run into equal
// parts for its warps, whatever heads they cross.  A warp keeps a reference, a sum and an output of the head it is in;
// they merge in shared memory, and a second kernel merges the parts of heads that several thread blocks share, in the
// order of the runs (no atomics: the same bits every time), and adds up the weights where they are gathered.
//
// A unit in a warp: codes come straight from global memory into registers in the layout of
// mma.m16n8k16's A operand -- keys (K) or head dimensions (V, transposed by byte permutes) as the
// 16 rows, the query rows as the 8 columns of B: few queries waste columns of a small MMA, not rows of a
// large one.  The order of d inside a dot product and of the output's d over MMA rows is free, so every
// lane reads 16 contiguous bytes at a time and no shared memory is involved.  S^T = K Q^T leaves
// weights whose 8x8 pieces movmatrix turns into the B operand of O^T += V^T P^T.  Codes are exact in fp16.
// The next unit's K is on its way while this one's V product runs, and the next V behind it.  (tcgen05 would
// take 128 keys a step and bring the 8 columns back through TMEM; the products are far from the bound.)
//
// A row's reference m moves only when a logit exceeds it by more than 2^kLazy, and V's scales are folded into the
// weights relative to a reference of their own, so the V product adds to the output in the MMA itself.  V's reference is
// a power of two and only rises (to a scale more than kRatio times as large), so the output in its units stays below 2^55:
// weights of 2^15, codes of 2^9, 2^31 keys.  A unit whose scale is more than kRatio times smaller, or all zeros, gets a
// product of its own that is added in fp32.  At a warp's end the output is divided by the sum before V's reference is
// applied, and merging takes weighted means: no answer passes fp32 that V's own numbers do not pass, however many keys.
//
// Roundings: q is scaled to fp16 by a power of two per row (bf16 has fewer bits: only
// elements 2^-25 of the row's largest are lost); the weights 2^8 e^(x - m) vscale / vref are rounded to fp16
// for the V product (2^-12 each, below the output's bf16; at most 2^15, and those under 2^-18 of the reference in
// steps of 2^-28 of it, so that 2^17 such keys together stay below 2^-12; it shows where their V is 2^18 times that of the
// keys that the row attends to), their sum is not.
//
// Measured (one B200, 8 KV heads of 128, 2 query heads each): 65537 keys 32.8 us, 4.1 TB/s of the 6.55 a copy reaches;
// about 10 us of every long step are fixed (launch and lengths 2.5, first loads 1.5, the last unit and the merge 2.5,
// the second kernel 3.7), the loads alone run at 5.8 TB/s, and the arithmetic without them takes half their time.  Two
// sequences of 131073 keys 92.5 us, 5.8 TB/s.  8705 keys 11.8 us (a cluster a head), 15.2 us with the weights.
#include <cmath>

#include "tg_cache.cuh"

namespace tg {
namespace q8 {

// Warps of a thread block, one a SM: 168 registers a thread for up to 8 query rows, 255 for 16.
constexpr int kDecWarps = 12;
__host__ __device__ constexpr int warps_of(int NT) { return NT == 1 ? kDecWarps : 8; }
constexpr int kMaxRows = 16;             // query rows per KV head
constexpr int kMaxCluster = 16;
constexpr int kMaxParts = 160;           // thread blocks of a launch that cuts the units into runs
constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;
constexpr float kShift = 8.0f * kLn2;    // weights are e^(x - m + kShift) ...
constexpr float kLazy = 3.0f * kLn2;     // ... at most 2^11 ...
constexpr float kRatio = 16.0f;          // ... times vscale / vref, at most kRatio, and not below 1 / kRatio in a joint product
constexpr float kNothing = -3.402823466e38f;   // the reference before the first logit
constexpr int kFinThreads = 256, kWeightKeys = 64, kWeightGroups = kFinThreads / kWeightKeys;
constexpr int kWeightTiles = kWeightGroups;   // tiles of keys at a time, one for each group to finish

struct DecodeArgs {
    Cache c;
    const __nv_bfloat16* q;
    const float* gain;
    __nv_bfloat16* out;
    float* lse;
    float scale;                         // tau / sqrt(d)
    int n_q, Hq, G, R;
    int Rp;                              // R rounded up to even: a key's logits in the workspace
    int cluster;                         // thread blocks of a head, as one cluster; 0: runs of units
    unsigned int* status;
    int2* heads;                         // [batch * Hkv] first thread block and number of the parts; 0 parts: done
    float2* rows;                        // [batch * Hkv][kMaxRows] reference and log2 of the sum, of heads that are done
    float* part;                         // [2 * grid][R][d]: means of a run's first / last head
    float2* part_ml;                     // [2 * grid][R]: their reference and sum
    float* logits;                       // [batch * Hkv][capacity][Rp]
};

// The two halves of a cluster barrier.
__device__ __forceinline__ void cluster_arrive() { asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory"); }
__device__ __forceinline__ void cluster_wait() { asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory"); }

__device__ __forceinline__ float ex2(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

__device__ __forceinline__ float exp_of(float x) { return ex2(x * kLog2e); }

template <int WORDS>
__device__ __forceinline__ void load_codes(const uint8_t* p, uint32_t* w) {
    if constexpr (WORDS == 4)
        asm volatile("ld.global.nc.L1::no_allocate.L2::128B.v4.u32 {%0,%1,%2,%3}, [%4];"
                     : "=r"(w[0]), "=r"(w[1]), "=r"(w[2]), "=r"(w[3])
                     : "l"(p));
    else
        asm volatile("ld.global.nc.L1::no_allocate.L2::128B.v2.u32 {%0,%1}, [%2];" : "=r"(w[0]), "=r"(w[1]) : "l"(p));
}

// D (16 x 8, fp32) += A (16 x 16) B (16 x 8), fp16.
__device__ __forceinline__ void mma(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                    uint32_t b1) {
    asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

__device__ __forceinline__ uint32_t transpose8x8(uint32_t x) {
    uint32_t y;
    asm("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
    return y;
}

__device__ __forceinline__ uint32_t pack_f16x2(float lo, float hi) {
    uint32_t r;
    asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
    return r;
}

// The registers of one unit: per lane g = lane / 4, t = lane % 4, the K codes of keys 8 r + g
// (r < 4), 16 bytes from 16 t of every 64; the V codes of keys 16 i + {2t, 2t + 1, 2t + 8, 2t + 9},
// d / 8 bytes from g d / 8; scales and biases.
template <int D>
struct KeyRegs {
    uint32_t w[4][D / 16];
    float scale, s[4];
};
template <int D>
struct ValueRegs {
    uint32_t w[2][4][D / 32];
    float scale;
};

template <int D, int FMT, int NT, bool kWeights>
struct Warp {
    const DecodeArgs& a;
    const int lane, g, t;
    uint32_t qf[D / 16][NT][2];
    float f[NT][2], gn[NT][2];          // logit factor and gain of this lane's query rows 8 nt + 2 t + {0, 1}
    float m[NT][2], l[NT][2], o[D / 16][NT][4];   // m: the reference less kShift
    float vinv;                          // o is in units of vref, a power of two; this is its inverse

    __device__ __forceinline__ explicit Warp(const DecodeArgs& args)
        : a(args), lane(threadIdx.x & 31), g(lane >> 2), t(lane & 3) {}

    // keys that the lane's row 8 nt + 2 t + c does not see at the sequence's end
    __device__ __forceinline__ int cut(int nt, int c) const {
        const int r = 8 * nt + 2 * t + c;
        return r < a.R ? a.n_q - 1 - r / a.G : 0;
    }

    // The query rows of one head: row r is query r / G, head kvh G + r % G.
    __device__ __forceinline__ void begin(int b, int kvh) {
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
            const int r = 8 * nt + g;
            uint4 u[D / 64][2];
            float amax = 0.0f;
            if (r < a.R) {
                const int64_t row =
                    (static_cast<int64_t>(b) * a.n_q + r / a.G) * a.Hq + static_cast<int64_t>(kvh) * a.G + r % a.G;
#pragma unroll
                for (int i = 0; i < D / 64; ++i) {
                    const uint4* p = reinterpret_cast<const uint4*>(a.q + row * D + 64 * i + 16 * t);
                    u[i][0] = __ldg(p);
                    u[i][1] = __ldg(p + 1);
                }
            } else {
#pragma unroll
                for (int i = 0; i < D / 64; ++i) u[i][0] = u[i][1] = make_uint4(0u, 0u, 0u, 0u);
            }
            float x[D / 64][16];
#pragma unroll
            for (int i = 0; i < D / 64; ++i) {
                const uint32_t w[8] = {u[i][0].x, u[i][0].y, u[i][0].z, u[i][0].w,
                                       u[i][1].x, u[i][1].y, u[i][1].z, u[i][1].w};
#pragma unroll
                for (int j = 0; j < 8; ++j) {
                    x[i][2 * j] = __uint_as_float(w[j] << 16);
                    x[i][2 * j + 1] = __uint_as_float(w[j] & 0xffff0000u);
                    amax = fmaxf(amax, fmaxf(fabsf(x[i][2 * j]), fabsf(x[i][2 * j + 1])));
                }
            }
            amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, 1));
            amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, 2));
            // 2^e <= amax < 2^(e + 1): q 2^-e is below 2 (rows with infinities stay as they are)
            int e = (__float_as_int(amax) >> 23) - 127;
            e = e > 127 ? 0 : max(min(e, 126), -126);
            const float down = __int_as_float((127 - e) << 23), up = __int_as_float((127 + e) << 23);
#pragma unroll
            for (int j = 0; j < D / 16; ++j) {
                const float* y = &x[j / 4][4 * (j % 4)];
                qf[j][nt][0] = pack_f16x2(y[0] * down, y[1] * down);
                qf[j][nt][1] = pack_f16x2(y[2] * down, y[3] * down);
            }
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                f[nt][i] = __shfl_sync(0xffffffffu, up, 4 * (2 * t + i)) * a.scale;
                const int rr = 8 * nt + 2 * t + i;
                gn[nt][i] = (rr < a.R && a.gain) ? __ldg(a.gain + kvh * a.G + rr % a.G) : 0.0f;
                m[nt][i] = kNothing;
                l[nt][i] = 0.0f;
            }
        }
#pragma unroll
        for (int dm = 0; dm < D / 16; ++dm)
#pragma unroll
            for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                for (int i = 0; i < 4; ++i) o[dm][nt][i] = 0.0f;
        vinv = inverse(__int_as_float(1 << 23));   // the least scale
    }

    __device__ __forceinline__ void load_keys(KeyRegs<D>& k, const uint8_t* p, const float* scale, const float* s) const {
#pragma unroll
        for (int r = 0; r < 4; ++r)
#pragma unroll
            for (int i = 0; i < D / 64; ++i) load_codes<4>(p + 8 * r * a.c.ld_token + 64 * i, &k.w[r][4 * i]);
        k.scale = __ldg(scale);
        if (a.c.s) {
#pragma unroll
            for (int r = 0; r < 4; ++r) k.s[r] = __ldg(s + 8 * r);
        }
    }
    __device__ __forceinline__ void load_values(ValueRegs<D>& v, const uint8_t* p, const float* scale) const {
#pragma unroll
        for (int i = 0; i < 2; ++i)
#pragma unroll
            for (int j = 0; j < 4; ++j)
                load_codes<D / 32>(p + (16 * i + (j & 1) + 8 * (j >> 1)) * a.c.ld_token, v.w[i][j]);
        v.scale = __ldg(scale);
    }

    // 1 / x for a power of two x in 2^-126 .. 2^126
    __device__ __forceinline__ static float inverse(float x) { return __int_as_float((254 << 23) - __float_as_int(x)); }

    // Whether a unit's product is added on its own: V's scale is far below the reference.
    __device__ __forceinline__ static bool apart(float ratio) { return ratio < 1.0f / kRatio; }

    // Weights of a unit as B operands, times V's scale over its reference (ratio; not where that is apart); the sums.
    __device__ __forceinline__ void scores(const KeyRegs<D>& k, float v_scale, int b, int kvh, int blk, int len,
                                           uint32_t (&pf)[2][NT][2], float& ratio) {
        float x[2][NT][4];
#pragma unroll
        for (int i = 0; i < 2; ++i) {
#pragma unroll
            for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                for (int c = 0; c < 4; ++c) x[i][nt][c] = 0.0f;
#pragma unroll
            for (int j = 0; j < D / 16; ++j) {
                const uint32_t a0 = decode2<FMT, false>(k.w[2 * i][j]), a2 = decode2<FMT, true>(k.w[2 * i][j]);
                const uint32_t a1 = decode2<FMT, false>(k.w[2 * i + 1][j]), a3 = decode2<FMT, true>(k.w[2 * i + 1][j]);
#pragma unroll
                for (int nt = 0; nt < NT; ++nt) mma(x[i][nt], a0, a1, a2, a3, qf[j][nt][0], qf[j][nt][1]);
            }
        }
        const bool bias = a.c.s && a.gain;
        if (bias) {
#pragma unroll
            for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                for (int i = 0; i < 2; ++i)
#pragma unroll
                    for (int c = 0; c < 4; ++c)
                        x[i][nt][c] = fmaf(x[i][nt][c], f[nt][c & 1] * k.scale, gn[nt][c & 1] * k.s[2 * i + (c >> 1)]);
        } else {
#pragma unroll
            for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                for (int i = 0; i < 2; ++i)
#pragma unroll
                    for (int c = 0; c < 4; ++c) x[i][nt][c] *= f[nt][c & 1] * k.scale;
        }
        if ((blk + 1) * kBlock > len - (a.n_q - 1)) {
#pragma unroll
            for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                for (int i = 0; i < 2; ++i)
#pragma unroll
                    for (int c = 0; c < 4; ++c)
                        if (blk * kBlock + 16 * i + 8 * (c >> 1) + g >= len - cut(nt, c & 1)) x[i][nt][c] = -INFINITY;
        }
        if constexpr (kWeights) {
#pragma unroll
            for (int nt = 0; nt < NT; ++nt)
                if (8 * nt + 2 * t < a.R) {
                    float* to = a.logits +
                                ((static_cast<int64_t>(b) * a.c.Hkv + kvh) * a.c.capacity + blk * kBlock + g) * a.Rp +
                                8 * nt + 2 * t;
#pragma unroll
                    for (int r = 0; r < 4; ++r)
                        *reinterpret_cast<float2*>(to + 8 * r * a.Rp) =
                            make_float2(x[r >> 1][nt][2 * (r & 1)],
                                        8 * nt + 2 * t + 1 < a.R ? x[r >> 1][nt][2 * (r & 1) + 1] : -INFINITY);
                }
        }
        // the lane's own largest logits against the reference: it rarely has to move
        bool move = false;
        float mx[NT][2];
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int c = 0; c < 2; ++c) {
                mx[nt][c] = fmaxf(fmaxf(x[0][nt][c], x[0][nt][c + 2]), fmaxf(x[1][nt][c], x[1][nt][c + 2]));
                move |= mx[nt][c] - m[nt][c] > kShift + kLazy;
            }
        if (__any_sync(0xffffffffu, move)) {
#pragma unroll
            for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                for (int c = 0; c < 2; ++c) {
                    float top = mx[nt][c];
#pragma unroll
                    for (int off = 4; off < 32; off <<= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, off));
                    const float mn = fmaxf(m[nt][c], top - kShift);
                    const float alpha = exp_of(m[nt][c] - mn);
                    m[nt][c] = mn;
                    l[nt][c] *= alpha;
#pragma unroll
                    for (int dm = 0; dm < D / 16; ++dm) {
                        o[dm][nt][c] *= alpha;
                        o[dm][nt][c + 2] *= alpha;
                    }
                }
        }
        ratio = v_scale * vinv;
        if (!(ratio <= kRatio)) {
            // far above V's reference: it rises to this scale's power of two (what is 2^149 below vanishes)
            const float up = inverse(__int_as_float(min(__float_as_int(v_scale) >> 23, 253) << 23));
            const float move = inverse(vinv) * up;
            vinv = up;
#pragma unroll
            for (int dm = 0; dm < D / 16; ++dm)
#pragma unroll
                for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                    for (int c = 0; c < 4; ++c) o[dm][nt][c] *= move;
            ratio = v_scale * vinv;
        }
        const float f = apart(ratio) ? 1.0f : ratio;
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                float p[4];
#pragma unroll
                for (int c = 0; c < 4; ++c) {
                    p[c] = exp_of(x[i][nt][c] - m[nt][c & 1]);
                    l[nt][c & 1] += p[c];
                }
                pf[i][nt][0] = transpose8x8(pack_f16x2(p[0] * f, p[1] * f));
                pf[i][nt][1] = transpose8x8(pack_f16x2(p[2] * f, p[3] * f));
            }
    }

    __device__ __forceinline__ void product(const ValueRegs<D>& v, int dm, const uint32_t (&pf)[2][NT][2],
                                            float (&acc)[NT][4]) const {
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            // bytes (key 2t, key 2t + 1) of head dimensions 2 dm and 2 dm + 1, and the same 8 keys on
            const uint32_t sel = dm & 1 ? 0x7362 : 0x5140;
            const uint32_t lo = __byte_perm(v.w[i][0][dm / 2], v.w[i][1][dm / 2], sel);
            const uint32_t hi = __byte_perm(v.w[i][2][dm / 2], v.w[i][3][dm / 2], sel);
            const uint32_t a0 = decode2<FMT, false>(lo), a1 = decode2<FMT, true>(lo);
            const uint32_t a2 = decode2<FMT, false>(hi), a3 = decode2<FMT, true>(hi);
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) mma(acc[nt], a0, a1, a2, a3, pf[i][nt][0], pf[i][nt][1]);
        }
    }
    __device__ __forceinline__ void values(ValueRegs<D>& v, int blk, int len, const uint32_t (&pf)[2][NT][2],
                                           float ratio, uint32_t& bad) {
        if (FMT == TG_CACHE_E4M3 && (blk + 1) * kBlock > len) {
            // rows behind the sequence may hold anything, NaN codes too: their weight is 0
#pragma unroll
            for (int i = 0; i < 2; ++i)
#pragma unroll
                for (int j = 0; j < 4; ++j)
                    if (blk * kBlock + 16 * i + 2 * t + (j & 1) + 8 * (j >> 1) >= len)
#pragma unroll
                        for (int w = 0; w < D / 32; ++w) v.w[i][j][w] = 0u;
        }
        if (FMT == TG_CACHE_E4M3 && unseen(blk, len)) {
            // nor may a NaN reach the queries that do not see its key (mark_nan sees to the others)
#pragma unroll
            for (int i = 0; i < 2; ++i)
#pragma unroll
                for (int j = 0; j < 4; ++j)
                    if (blk * kBlock + 16 * i + 2 * t + (j & 1) + 8 * (j >> 1) >= len - (a.n_q - 1))
#pragma unroll
                        for (int w = 0; w < D / 32; ++w) {
                            const uint32_t nan = nan_bytes(v.w[i][j][w]);
                            bad |= nan;
                            v.w[i][j][w] &= ~nan;
                        }
        }
        if (apart(ratio)) {
#pragma unroll
            for (int dm = 0; dm < D / 16; ++dm) {
                float acc[NT][4] = {};
                product(v, dm, pf, acc);
#pragma unroll
                for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                    for (int c = 0; c < 4; ++c) o[dm][nt][c] = fmaf(acc[nt][c], ratio, o[dm][nt][c]);
            }
        } else {
#pragma unroll
            for (int dm = 0; dm < D / 16; ++dm) product(v, dm, pf, o[dm]);
        }
    }

    // Whether a block has keys that some query sees and some does not.
    __device__ __forceinline__ bool unseen(int blk, int len) const {
        return a.n_q > 1 && (blk + 1) * kBlock > len - (a.n_q - 1);
    }
    __device__ __forceinline__ static uint32_t nan_bytes(uint32_t codes) { return __vcmpeq4(codes & 0x7f7f7f7fu, 0x7f7f7f7fu); }
    // NaN in the outputs of the queries that see a key with a NaN in V, of a block with keys that not all see: where the product
    // of the NaN codes' places (1 or 0) with what each row sees is not 0.
    __device__ __forceinline__ void mark_nan(ValueRegs<D>& v, int blk, int len) {
        const int last = len - blk * kBlock;
#pragma unroll
        for (int i = 0; i < 2; ++i)
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const int key = 16 * i + 2 * t + (j & 1) + 8 * (j >> 1);
#pragma unroll
                for (int w = 0; w < D / 32; ++w)   // e4m3's 1
                    v.w[i][j][w] = key >= last - (a.n_q - 1) && key < last ? nan_bytes(v.w[i][j][w]) & 0x38383838u : 0u;
            }
        uint32_t seen[2][NT][2];             // as B operands: 1 where row 8 nt + g sees the key
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
            const int r = 8 * nt + g, end = last - (r < a.R ? a.n_q - 1 - r / a.G : 0) - 2 * t;
#pragma unroll
            for (int i = 0; i < 2; ++i)
#pragma unroll
                for (int k = 0; k < 2; ++k)
                    seen[i][nt][k] = (16 * i + 8 * k < end ? 0x3c00u : 0u) | (16 * i + 8 * k + 1 < end ? 0x3c000000u : 0u);
        }
#pragma unroll
        for (int dm = 0; dm < D / 16; ++dm) {
            float acc[NT][4] = {};
            product(v, dm, seen, acc);
#pragma unroll
            for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                for (int c = 0; c < 4; ++c)
                    if (acc[nt][c] > 0.0f) o[dm][nt][c] = __int_as_float(0x7fffffff);
        }
    }

    // Units u0, u0 + step, ... < u1 of one head.
    __device__ __forceinline__ void run(int b, int kvh, int u0, int u1, int step, int len) {
        const int64_t block_codes = kBlock * a.c.ld_token, codes = b * a.c.ld_seq + u0 * block_codes + kvh * D;
        const uint8_t* pk = a.c.k + codes + g * a.c.ld_token + 16 * t;
        const uint8_t* pv = a.c.v + codes + 2 * t * a.c.ld_token + g * (D / 8);
        const int64_t scale = (b * a.c.blocks() + u0) * a.c.Hkv + kvh;
        const float *ks = a.c.k_scale + scale, *vs = a.c.v_scale + scale;
        const float* s = a.c.s + b * a.c.capacity + u0 * kBlock + g;   // (used where there is an s)
        KeyRegs<D> k;
        ValueRegs<D> v;
        if (u0 < u1) {
            load_keys(k, pk, ks, s);
            load_values(v, pv, vs);
        }
        begin(b, kvh);
        uint32_t bad = 0;
        int u = u0;
        for (; u < u1; u += step) {
            uint32_t pf[2][NT][2];
            float ratio;
            scores(k, v.scale, b, kvh, u, len, pf, ratio);
            pk += step * block_codes;
            pv += step * block_codes;
            ks += step * a.c.Hkv;
            vs += step * a.c.Hkv;
            s += step * kBlock;
            if (u + step < u1) load_keys(k, pk, ks, s);
            values(v, u, len, pf, ratio, bad);
            if (u + step < u1) load_values(v, pv, vs);
        }
        if (FMT == TG_CACHE_E4M3 && __any_sync(0xffffffffu, bad)) {
            // among the last 2 blocks of the sequence (one that is another warp's may be marked twice)
#pragma unroll 1
            for (int i = 0; i < 2; ++i) {
                u -= step;
                if (u < 0 || !unseen(u, len)) continue;
                load_values(v, a.c.v + b * a.c.ld_seq + (u * static_cast<int64_t>(kBlock) + 2 * t) * a.c.ld_token + kvh * D + g * (D / 8),
                            a.c.v_scale + (b * a.c.blocks() + u) * a.c.Hkv + kvh);
                mark_nan(v, u, len);
            }
        }
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int c = 0; c < 2; ++c)
#pragma unroll
                for (int off = 4; off < 32; off <<= 1) l[nt][c] += __shfl_xor_sync(0xffffffffu, l[nt][c], off);
    }
};

// The reference and log2 of the sum of a row (infinity where there is no weight), and the row's log-sum-exp.
__device__ __forceinline__ float2 row_of(float m, float l) { return make_float2(m, l == 0.0f ? INFINITY : log2f(l)); }
__device__ __forceinline__ float lse_of(float2 row) { return row.y == INFINITY ? -INFINITY : fmaf(row.y, kLn2, row.x); }
__device__ __forceinline__ int64_t out_row(const DecodeArgs& a, int b, int kvh, int r) {
    return (static_cast<int64_t>(b) * a.n_q + r / a.G) * a.Hq + kvh * a.G + r % a.G;
}
// 1 / l of a sum of weights (below 2^11 * 2^31); 0 where there is no key, or none above -inf.
__device__ __forceinline__ float share(float l) { return l == 0.0f ? 0.0f : __fdividef(1.0f, l); }
// Four outputs of one row.
__device__ __forceinline__ void store_out(__nv_bfloat16* to, float4 o) {
    *reinterpret_cast<uint2*>(to) = make_uint2(pack_bf16x2(o.x, o.y), pack_bf16x2(o.z, o.w));
}
__device__ __forceinline__ void add4(float4& o, const float4& x, float f) {
    o.x = fmaf(x.x, f, o.x);
    o.y = fmaf(x.y, f, o.y);
    o.z = fmaf(x.z, f, o.z);
    o.w = fmaf(x.w, f, o.w);
}

__device__ __forceinline__ void finish_row(const DecodeArgs& a, int b, int kvh, int r, int d, int D, float m, float l,
                                           float4 o) {
    store_out(a.out + out_row(a, b, kvh, r) * D + d, o);
    if (d != 0) return;
    const float2 row = row_of(m, l);
    a.rows[(static_cast<int64_t>(b) * a.c.Hkv + kvh) * kMaxRows + r] = row;
    if (a.lse) a.lse[out_row(a, b, kvh, r)] = lse_of(row);
}

// A thread block's part of one head.
struct Segment {
    int b, kvh, len;
    unsigned from, to;                   // its units, counted from the run's first
    int u0;                              // the first of them in the head
    int e0, e1;                          // the entries of the warps' sums (below) that are its
    int parts;                           // thread blocks that share the head
    int slot;                            // this thread block's part
};

// A warp's means (o), references and sums of the segment it is in: the warps' parts and the segments are in the same order,
// so those of warp w and segment j are entry w + j.
template <int D, int NT>
struct Shared {
    static constexpr int kW = warps_of(NT);
    float o[2 * kW][8 * NT][D];
    float m[2 * kW][8 * NT], l[2 * kW][8 * NT];
    Segment seg[kW];
    unsigned red[kW], base, next, total;
    int n_seg, b;
    // what the thread blocks of a cluster hand to the one that finishes a number: their means, references and sums
    float4 means[8 * NT * D / 4 + kMaxCluster];
    float2 ml[kMaxCluster][8 * NT];
};

template <int D, int FMT, int NT, bool kWeights>
__device__ __forceinline__ void keep_sums(const DecodeArgs& a, Shared<D, NT>& sh,
                                          const Warp<D, FMT, NT, kWeights>& wp, int entry) {
    const float vref = wp.inverse(wp.vinv);
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int c = 0; c < 2; ++c) {
            const int r = 8 * nt + 2 * wp.t + c;
            if (wp.g == 0) {
                sh.m[entry][r] = wp.m[nt][c];
                sh.l[entry][r] = wp.l[nt][c];
            }
            if (r < a.R) {
                const float part = share(wp.l[nt][c]);
                float* to = &sh.o[entry][r][D / 8 * wp.g];
#pragma unroll
                for (int dm = 0; dm < D / 16; ++dm)
                    *reinterpret_cast<float2*>(to + 2 * dm) =
                        make_float2(wp.o[dm][nt][c] * part * vref, wp.o[dm][nt][2 + c] * part * vref);
            }
        }
}

__device__ __forceinline__ void store_cluster(void* to, uint32_t rank, float4 v) {
    asm volatile("st.shared::cluster.v4.f32 [%0], {%1, %2, %3, %4};" ::"r"(cluster_addr(to, rank)), "f"(v.x), "f"(v.y),
                 "f"(v.z), "f"(v.w)
                 : "memory");
}
__device__ __forceinline__ void store_cluster(void* to, uint32_t rank, float2 v) {
    asm volatile("st.shared::cluster.v2.f32 [%0], {%1, %2};" ::"r"(cluster_addr(to, rank)), "f"(v.x), "f"(v.y) : "memory");
}

// Merges the warps' means of the block's segments: whole heads are done, the others' parts go to the workspace, or, in
// a cluster, to the thread block that finishes them (float4 i of the head is block i % cluster's).
template <int D, int NT>
__device__ __forceinline__ void merge_warps(const DecodeArgs& a, Shared<D, NT>& sh, int n_seg) {
    constexpr int kW = warps_of(NT);
    __syncthreads();
    for (int i = threadIdx.x; i < n_seg * a.R * (D / 4); i += kW * 32) {
        const int jr = i / (D / 4), j = jr / a.R, r = jr % a.R, d = i % (D / 4) * 4;
        const Segment& sg = sh.seg[j];
        const int e0 = sg.e0, n = sg.e1 - e0;   // n < kW
        float f[kW], le[kW], m = kNothing, l = 0.0f;
        unsigned live = 0;                   // the warps with units: the others left no means
#pragma unroll
        for (int e = 0; e < kW; ++e) {
            f[e] = e <= n ? sh.m[e0 + e][r] : -INFINITY;
            le[e] = e <= n ? sh.l[e0 + e][r] : 0.0f;
            live |= f[e] == -INFINITY ? 0u : 1u << e;
            m = fmaxf(m, f[e]);
        }
#pragma unroll
        for (int e = 0; e < kW; ++e) {
            f[e] = exp_of(f[e] - m);
            l = fmaf(le[e], f[e], l);
        }
        const float part = share(l);
        float4 o = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
#pragma unroll
        for (int e = 0; e < kW; ++e)
            // (a warp that saw no key above -inf adds 0, or the NaN of a value: every launch gives the same)
            if (live >> e & 1u) add4(o, *reinterpret_cast<const float4*>(&sh.o[e0 + e][r][d]), le[e] * f[e] * part);
        if (a.cluster > 1) {
            const int v = r * (D / 4) + d / 4, rank = cluster_rank_in(), each = (a.R * (D / 4) - 1) / a.cluster + 1;
            store_cluster(&sh.means[rank * each + v / a.cluster], v % a.cluster, o);
            if (d / 4 < a.cluster) store_cluster(&sh.ml[rank][r], d / 4, make_float2(m, l));
        } else if (sg.parts == 1) {
            finish_row(a, sg.b, sg.kvh, r, d, D, m, l, o);
        } else {
            *reinterpret_cast<float4*>(a.part + (static_cast<int64_t>(sg.slot) * a.R + r) * D + d) = o;
            if (d == 0) a.part_ml[sg.slot * a.R + r] = make_float2(m, l);
        }
    }
}

template <int D, int FMT, int NT, bool kWeights>
__global__ void __launch_bounds__(warps_of(NT) * 32, 1) gated_decode_q8_kernel(const DecodeArgs a) {
    constexpr int kW = warps_of(NT), kThreads = kW * 32;
    extern __shared__ __align__(16) uint8_t smem[];
    Shared<D, NT>& sh = *reinterpret_cast<Shared<D, NT>*>(smem);
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    if (a.cluster > 1) cluster_arrive();
    pdl_wait();
    pdl_trigger();
    const int B = a.c.batch, Hkv = a.c.Hkv;
    Warp<D, FMT, NT, kWeights> wp(a);

    if (a.cluster) {
        const int head = blockIdx.x / a.cluster, rank = blockIdx.x % a.cluster, b = head / Hkv, kvh = head % Hkv;
        const int len = length_of(a.c, b, a.status);
        if (tid == 0) {
            sh.seg[0] = Segment{b, kvh, len, 0u, 0u, 0, 0, kW - 1, 1, 0};
            if (rank == 0) a.heads[head] = make_int2(0, 0);
        }
        wp.run(b, kvh, rank * kW + warp, (len + kBlock - 1) / kBlock, a.cluster * kW, len);
        keep_sums<D, FMT, NT, kWeights>(a, sh, wp, warp);
        __syncwarp();
        if (a.cluster > 1) cluster_wait();   // every thread block of the cluster has begun
        merge_warps<D, NT>(a, sh, 1);
        if (a.cluster > 1) {
            __syncwarp();
            cluster_sync_all();
            const int vecs = a.R * (D / 4), each = (vecs - 1) / a.cluster + 1;
            for (int i = tid; i * a.cluster + rank < vecs; i += kThreads) {
                const int v = i * a.cluster + rank, r = v / (D / 4), d = v % (D / 4) * 4;
                float m = kNothing, l = 0.0f;
                for (int p = 0; p < a.cluster; ++p) m = fmaxf(m, sh.ml[p][r].x);
#pragma unroll 4
                for (int p = 0; p < a.cluster; ++p) l = fmaf(sh.ml[p][r].y, exp_of(sh.ml[p][r].x - m), l);
                const float part = share(l);
                float4 o = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
#pragma unroll 4
                for (int p = 0; p < a.cluster; ++p) {
                    const float2 ml = sh.ml[p][r];
                    add4(o, sh.means[p * each + i], ml.y * exp_of(ml.x - m) * part);
                }
                finish_row(a, b, kvh, r, d, D, m, l, o);
            }
        }
        return;
    }

    // All units (a unit is 4 KB of memory at least: their number fits 32 bits), this thread block's
    // run of them and the sequence in which it begins; base: units before that sequence.
    auto units_of = [&](int b) -> unsigned {
        return static_cast<unsigned>((length_of(a.c, b, a.status) + kBlock - 1) / kBlock) * Hkv;
    };
    auto scan = [&](unsigned mine, unsigned& before) -> unsigned {   // exclusive scan, returns the sum
        unsigned incl = mine;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const unsigned y = __shfl_up_sync(0xffffffffu, incl, o);
            if (lane >= o) incl += y;
        }
        if (lane == 31) sh.red[warp] = incl;
        __syncthreads();
        unsigned all = 0;
        before = incl - mine;
#pragma unroll
        for (int w = 0; w < kW; ++w) {
            before += w < warp ? sh.red[w] : 0u;
            all += sh.red[w];
        }
        __syncthreads();
        return all;
    };
    unsigned total = 0, mine = 0, before = 0;
    if (B == 1) {
        total = units_of(0);
    } else {
        for (int b0 = 0; b0 < B; b0 += kThreads) {
            mine = b0 + tid < B ? units_of(b0 + tid) : 0u;
            total += scan(mine, before);
        }
    }
    const unsigned n = gridDim.x < total ? gridDim.x : total;   // thread blocks with work
    unsigned u = 0, u_end = 0;
    if (blockIdx.x < n) {
        u = static_cast<unsigned>(static_cast<uint64_t>(total) * blockIdx.x / n);
        u_end = static_cast<unsigned>(static_cast<uint64_t>(total) * (blockIdx.x + 1) / n);
    }
    if (tid == 0) sh.total = total;
    if (B > 1 && u < u_end) {
        unsigned base = 0;
        for (int b0 = 0;; b0 += kThreads) {
            if (B > kThreads) {       // (a single round of sequences is still in registers)
                mine = b0 + tid < B ? units_of(b0 + tid) : 0u;
                const unsigned sum = scan(mine, before);
                before += base;
                base += sum;
            } else {
                __syncthreads();
                base = total;
            }
            if (before <= u && u < before + mine) {
                sh.b = b0 + tid;
                sh.base = before;
            }
            if (u < base) break;
        }
        __syncthreads();
    }

    while (u < u_end) {
        // The next segments of the run, as many as there are warps.  One sequence's follow from its length; others
        // are looked up by one thread.
        if (B == 1) {
            const int len = length_of(a.c, 0, a.status);
            const unsigned nblk = (len + kBlock - 1) / kBlock, h = u / nblk + tid, last = (u_end - 1) / nblk;
            if (tid < kW && h <= last) {
                const unsigned head = h * nblk, from = max(head, u), to = min(head + nblk, u_end);
                sh.seg[tid] = Segment{0, static_cast<int>(h), len, from - u, to - u, static_cast<int>(from - head)};
                if (tid == kW - 1 || h == last) {
                    sh.n_seg = tid + 1;
                    sh.next = to;
                }
            }
        } else if (tid == 0) {
            int k = 0, b = sh.b;
            unsigned base = sh.base, v = u;
            while (v < u_end && k < kW) {
                const int len = length_of(a.c, b, a.status);
                const unsigned nblk = (len + kBlock - 1) / kBlock;
                if (nblk == 0) {         // nothing here: the next sequence
                    ++b;
                    continue;
                }
                const unsigned kvh = (v - base) / nblk, head = base + kvh * nblk, to = min(head + nblk, u_end);
                sh.seg[k] = Segment{b, static_cast<int>(kvh), len, v - u, to - u, static_cast<int>(v - head)};
                ++k;
                v = to;
                if (v == head + nblk && kvh == static_cast<unsigned>(Hkv) - 1) {
                    base += nblk * Hkv;
                    ++b;
                }
            }
            sh.n_seg = k;
            sh.b = b;
            sh.base = base;
            sh.next = v;
        }
        __syncthreads();
        {
            // this warp's units of the run
            const unsigned units = sh.next - u;
            unsigned x = units * warp / kW;
            const unsigned x_end = units * (warp + 1) / kW;
            int j = 0;
            while (j + 1 < sh.n_seg && x >= sh.seg[j].to) ++j;
            if (x == x_end && lane < 8 * NT) sh.m[warp + j][lane] = -INFINITY, sh.l[warp + j][lane] = 0.0f;
            for (; x < x_end; ++j) {
                const Segment& sg = sh.seg[j];
                const unsigned stop = min(sg.to, x_end);
                const int u0 = sg.u0 + static_cast<int>(x - sg.from);
                wp.run(sg.b, sg.kvh, u0, u0 + static_cast<int>(stop - x), 1, sg.len);
                keep_sums<D, FMT, NT, kWeights>(a, sh, wp, warp + j);
                x = stop;
            }
        }
        const int n_seg = sh.n_seg;
        if (tid < n_seg) {
            // the thread blocks with the head's first and last unit, the warps with the segment's
            Segment& sg = sh.seg[tid];
            const unsigned units = sh.next - u, nblk = (sg.len + kBlock - 1) / kBlock, head = u + sg.from - sg.u0;
            const unsigned total = sh.total, n = min(gridDim.x, total);
            const int i0 = static_cast<int>(((head + 1ull) * n - 1) / total);
            const int i1 = static_cast<int>((static_cast<uint64_t>(head + nblk) * n - 1) / total);
            sg.parts = i1 - i0 + 1;
            sg.slot = 2 * blockIdx.x + (i0 == static_cast<int>(blockIdx.x) ? 1 : 0);
            if (sg.u0 == 0) a.heads[sg.b * Hkv + sg.kvh] = make_int2(i0, i0 == i1 ? 0 : i1 - i0 + 1);
            sg.e0 = tid + static_cast<int>(((sg.from + 1) * kW - 1) / units);
            sg.e1 = tid + static_cast<int>((sg.to * kW - 1) / units);
        }
        merge_warps<D, NT>(a, sh, n_seg);
        u = sh.next;
        __syncthreads();
    }

    // sequences without a token have no units: their rows are 0
    for (int e = blockIdx.x; e < B; e += gridDim.x) {
        if (length_of(a.c, e, a.status) > 0) continue;
        for (int i = tid; i < a.n_q * a.Hq * D; i += kThreads)
            a.out[static_cast<int64_t>(e) * a.n_q * a.Hq * D + i] = __float2bfloat16_rn(0.0f);
        for (int i = tid; i < a.n_q * a.Hq; i += kThreads)
            if (a.lse) a.lse[static_cast<int64_t>(e) * a.n_q * a.Hq + i] = -INFINITY;
        for (int i = tid; i < Hkv; i += kThreads) a.heads[e * Hkv + i] = make_int2(0, 0);
    }
}

// Room of a thread block of the second kernel, for either of its tasks.
constexpr int kMergeVecs = 64, kMergeGroups = kFinThreads / kMergeVecs;   // float4s of the output a thread block merges
struct MergeRoom {
    float f[kMaxParts][4];               // the parts' shares of its 2 or 4 rows
    float4 sum[kMergeGroups][kMergeVecs];
};
struct WeightRoom {
    float2 rows[64 * kMaxRows];          // as row_of makes them; the odd last row adds nothing
    float sum[kWeightTiles][kWeightGroups][kWeightKeys];
};

// Merges the parts of one head that several thread blocks shared, in the order of the parts: rows r0, r0 + 1, ... (2 of
// 128 or 4 of 64 numbers).  Groups of threads take the parts in turn; the first of them are under way while the factors
// form.
template <int D>
__device__ __forceinline__ void merge_parts(const DecodeArgs& a, MergeRoom& room, int b, int h, int r0) {
    constexpr int kRows = kMergeVecs / (D / 4), kAhead = 6, kPer = kMaxParts / 32;
    const int tid = threadIdx.x, i = tid % kMergeVecs, grp = tid / kMergeVecs, r = i / (D / 4), d = i % (D / 4) * 4;
    // part p of a head belongs to thread block hd.x + p: its last head for p = 0, its first one otherwise
    const int2 hd = a.heads[b * a.c.Hkv + h];
    auto slot = [&](int p) -> int64_t { return 2 * (hd.x + p) + (p == 0); };
    const int np = hd.y;
    if (np == 0) return;
    const bool active = r0 + r < a.R;
    const float* from = a.part + (r0 + r) * D + d;
    float4 x[kAhead];
    auto load = [&](int p0) {
#pragma unroll
        for (int y = 0; y < kAhead; ++y) {
            const int p = p0 + y * kMergeGroups;
            if (active && p < np) x[y] = __ldcg(reinterpret_cast<const float4*>(from + slot(p) * a.R * D));
        }
    };
    load(grp);
    const int row = r0 + tid / 32;        // one warp a row
    if (tid / 32 < kRows && row < a.R) {
        float2 ml[kPer];
        float m = kNothing, l = 0.0f;
#pragma unroll
        for (int y = 0; y < kPer; ++y) {
            const int p = tid % 32 + 32 * y;
            ml[y] = p < np ? __ldcg(a.part_ml + slot(p) * a.R + row) : make_float2(kNothing, 0.0f);
            m = fmaxf(m, ml[y].x);
        }
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
#pragma unroll
        for (int y = 0; y < kPer; ++y) {
            ml[y].y *= exp_of(ml[y].x - m);
            l += ml[y].y;
        }
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) l += __shfl_xor_sync(0xffffffffu, l, o);
        const float part = share(l);
#pragma unroll
        for (int y = 0; y < kPer; ++y)
            if (tid % 32 + 32 * y < np) room.f[tid % 32 + 32 * y][tid / 32] = ml[y].y * part;
        if (tid % 32 == 0 && a.lse) a.lse[out_row(a, b, h, row)] = lse_of(row_of(m, l));
    }
    __syncthreads();
    float4 o = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
    for (int p0 = grp; p0 < np; p0 += kAhead * kMergeGroups) {
        if (p0 > grp) load(p0);
#pragma unroll
        for (int y = 0; y < kAhead; ++y) {
            const int p = p0 + y * kMergeGroups;
            if (active && p < np) add4(o, x[y], room.f[p][r]);
        }
    }
    room.sum[grp][i] = o;
    __syncthreads();
    if (grp == 0 && active) {
#pragma unroll
        for (int y = 1; y < kMergeGroups; ++y) add4(o, room.sum[y][i], 1.0f);
        store_out(a.out + out_row(a, b, h, r0 + r) * D + d, o);
    }
}

// The weights of keys x * 64, ..., VEC rows of a head at a time.
template <int VEC>
__device__ __forceinline__ void add_tiles(const DecodeArgs& a, WeightRoom& room, int b, int x, int nx, int len) {
    const int tid = threadIdx.x, key = tid % kWeightKeys, grp = tid / kWeightKeys;
    const int vecs = a.Rp / VEC, items = a.c.Hkv * vecs;
    const int64_t stride = static_cast<int64_t>(nx) * kWeightKeys;
    for (int64_t c0 = static_cast<int64_t>(x) * kWeightKeys; c0 < len; c0 += kWeightTiles * stride) {
        const int64_t c = c0 + key + grp * stride;   // each group finishes one tile
        float* to = a.c.w + b * a.c.capacity + c;
        const float before = c < len ? *to : 0.0f;
        float sum[kWeightTiles] = {};
        const float* from = a.logits + (static_cast<int64_t>(b) * a.c.Hkv * a.c.capacity + c0 + key) * a.Rp;
#pragma unroll 2
        for (int i = grp; i < items; i += kWeightGroups) {
            const int h = i / vecs, r = (i - h * vecs) * VEC;
            const float* p = from + h * a.c.capacity * a.Rp + r;
            float2 row[VEC];
#pragma unroll
            for (int q = 0; q < VEC; ++q) row[q] = room.rows[h * a.Rp + r + q];
#pragma unroll
            for (int j = 0; j < kWeightTiles; ++j)
                if (c0 + key + j * stride < len) {
                    float y[VEC];
                    if constexpr (VEC == 4)
                        *reinterpret_cast<float4*>(y) = __ldcg(reinterpret_cast<const float4*>(p + j * stride * a.Rp));
                    else
                        *reinterpret_cast<float2*>(y) = __ldcg(reinterpret_cast<const float2*>(p + j * stride * a.Rp));
#pragma unroll
                    for (int q = 0; q < VEC; ++q) sum[j] += ex2(fmaf(y[q] - row[q].x, kLog2e, -row[q].y));
                }
        }
#pragma unroll
        for (int j = 0; j < kWeightTiles; ++j) room.sum[j][grp][key] = sum[j];
        __syncthreads();
        if (c < len) {
            float total = 0.0f;
#pragma unroll
            for (int i = 0; i < kWeightGroups; ++i) total += room.sum[grp][i][key];
            *to = before + total;
        }
        __syncthreads();
    }
}

// w[b, c] += sum over heads and rows of e^(x - m) / l, thread block x of nx: 64 keys and 4 groups of heads, up to 4 tiles
// of keys at once so that many loads are under way, the groups' sums in a fixed order.  The log-sum-exps come from
// the parts themselves, so that this does not wait for their merging.
__device__ __forceinline__ void add_weights(const DecodeArgs& a, WeightRoom& room, int b, int x, int nx, bool done) {
    const int tid = threadIdx.x, Hkv = a.c.Hkv, len = length_of(a.c, b, a.status);
    if (static_cast<int64_t>(x) * kWeightKeys >= len) return;
    if (done) {
        // every head's rows are finished already
        for (int i = tid; i < Hkv * a.Rp; i += kFinThreads) {
            const int h = i / a.Rp, r = i - h * a.Rp;
            room.rows[i] = r < a.R ? a.rows[(static_cast<int64_t>(b) * Hkv + h) * kMaxRows + r] : row_of(0.0f, 0.0f);
        }
    }
    // else 8 lanes a row
    for (int i = tid / 8; !done && i < (Hkv * a.Rp + 3) / 4 * 4; i += kFinThreads / 8) {
        const int h = i / a.Rp, r = i % a.Rp;
        const bool row = h < Hkv && r < a.R;
        const int2 hd = row ? a.heads[b * Hkv + h] : make_int2(0, 0);
        float2 v = row && hd.y == 0 ? a.rows[(static_cast<int64_t>(b) * Hkv + h) * kMaxRows + r] : row_of(0.0f, 0.0f);
        float m = kNothing, l = 0.0f;
        for (int p0 = tid % 8; p0 < hd.y; p0 += 32) {
            float2 ml[4];
#pragma unroll
            for (int y = 0; y < 4; ++y) {
                const int p = p0 + 8 * y;
                ml[y] = p < hd.y ? __ldcg(a.part_ml + (2 * (hd.x + p) + (p == 0)) * a.R + r) : make_float2(kNothing, 0.0f);
            }
            const float mn = fmaxf(fmaxf(m, fmaxf(ml[0].x, ml[1].x)), fmaxf(ml[2].x, ml[3].x));
            l *= exp_of(m - mn);
#pragma unroll
            for (int y = 0; y < 4; ++y) l = fmaf(ml[y].y, exp_of(ml[y].x - mn), l);
            m = mn;
        }
#pragma unroll
        for (int o = 4; o > 0; o >>= 1) {
            const float m2 = __shfl_xor_sync(0xffffffffu, m, o), l2 = __shfl_xor_sync(0xffffffffu, l, o);
            const float mn = fmaxf(m, m2);
            l = l * exp_of(m - mn) + l2 * exp_of(m2 - mn);
            m = mn;
        }
        if (hd.y) v = row_of(m, l);
        if (tid % 8 == 0 && h < Hkv) room.rows[i] = v;
    }
    __syncthreads();
    if (a.Rp % 4 == 0)
        add_tiles<4>(a, room, b, x, nx, len);
    else
        add_tiles<2>(a, room, b, x, nx, len);
}

// The second kernel: thread blocks x < merges of sequence b merge its heads' rows, the others add up its weights.
template <int D>
__global__ void __launch_bounds__(kFinThreads, 4) decode_q8_finish_kernel(const DecodeArgs a, int merges) {
    __shared__ union __align__(16) Room {
        MergeRoom merge;
        WeightRoom weights;
        __device__ Room() {}
    } room;
    pdl_wait();
    pdl_trigger();
    const int x = blockIdx.x, b = blockIdx.y;
    constexpr int kRows = kMergeVecs / (D / 4);
    const int chunks = (a.R + kRows - 1) / kRows;
    if (x < merges)
        merge_parts<D>(a, room.merge, b, x / chunks, x % chunks * kRows);
    else
        add_weights(a, room.weights, b, x - merges, gridDim.x - merges, merges == 0);
}

// Workspace: status header, heads, rows, parts, logits (each from a 256-byte boundary).
struct Layout {
    size_t heads, rows, part, part_ml, logits, bytes;
};
static size_t up256(size_t x) { return (x + 255) / 256 * 256; }
static Layout layout(const Cache& c, int d_h, int R, bool weights) {
    const int64_t heads = static_cast<int64_t>(c.batch) * c.Hkv;
    Layout L;
    L.heads = kWsHeader;
    L.rows = L.heads + up256(static_cast<size_t>(heads) * 8);
    L.part = L.rows + up256(static_cast<size_t>(heads) * kMaxRows * 8);
    L.part_ml = L.part + up256(static_cast<size_t>(2 * kMaxParts) * R * d_h * 4);
    L.logits = L.part_ml + up256(static_cast<size_t>(2 * kMaxParts) * R * 8);
    L.bytes = L.logits + (weights ? up256(static_cast<size_t>(heads) * c.capacity * ((R + 1) / 2 * 2) * 4) : 0);
    return L;
}

// Clusters of `cl` thread blocks that run at the same time (0: none fits), asked for once per kernel and device.
template <int D, int FMT, int NT, bool kWeights>
static int max_clusters(int cl) {
    static std::atomic<int> cache[64][kMaxCluster + 1];
    const int dev = current_device();
    if (dev >= 0 && cache[dev][cl].load(std::memory_order_acquire)) return cache[dev][cl].load() - 1;
    auto kern = gated_decode_q8_kernel<D, FMT, NT, kWeights>;
    constexpr int kSmem = static_cast<int>(sizeof(Shared<D, NT>));
    int n = 0;
    if (cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmem) == cudaSuccess &&
        (cl <= 8 || cudaFuncSetAttribute(kern, cudaFuncAttributeNonPortableClusterSizeAllowed, 1) == cudaSuccess)) {
        cudaLaunchConfig_t cfg = {};
        cfg.gridDim = dim3(static_cast<unsigned>(cl));
        cfg.blockDim = dim3(warps_of(NT) * 32);
        cfg.dynamicSmemBytes = kSmem;
        cudaLaunchAttribute at[1];
        at[0].id = cudaLaunchAttributeClusterDimension;
        at[0].val.clusterDim.x = static_cast<unsigned>(cl);
        at[0].val.clusterDim.y = at[0].val.clusterDim.z = 1;
        cfg.attrs = at;
        cfg.numAttrs = 1;
        if (cudaOccupancyMaxActiveClusters(&n, kern, &cfg) != cudaSuccess) {
            cudaGetLastError();
            n = 0;
        }
    } else {
        cudaGetLastError();
    }
    if (dev >= 0) cache[dev][cl].store(n + 1, std::memory_order_release);
    return n;
}

// Thread blocks of a head: the fewest that give a warp no more units than the most whose clusters all run at the same
// time would, one unit where that many fit; 0 (runs of units) where a warp would have more than 2 units in a thread
// block alone, or 4 in a cluster.  Returns -1 where the kernel cannot be set up.  Measured, e4m3 without weights, cluster
// against runs in us (* the side that the rule takes):
//   keys                       1025       2049        4097         8705        12289        16385        24577        65537
//   8 heads of 2 rows      *7.7  9.4  *7.3  9.9   *9.5 10.1   *11.3 12.5   *13.6 14.7   *16.3 16.1   20.6 *19.0   40.0 *32.6
//   16 heads of 2 rows     *7.9 10.1  *7.7 10.3  *10.6 13.4   *14.9 17.3   19.0 *19.8   22.8 *21.9   28.8 *26.8   62.5 *52.5
//   one head of 8 rows     *7.9  9.4  *7.5 10.4   *8.1 13.3    *9.6 13.0   *11.0 13.2   *11.3 13.4   14.1 *13.7   25.0 *17.3
// (16 heads over 2049 keys take 9.7 us where only powers of two are allowed as a cluster's size.)
template <int D, int FMT, int NT, bool kWeights>
static int cluster_for(int64_t heads, int64_t blocks) {
    static std::atomic<int> smem_set[64];
    if (!set_max_dynamic_smem(gated_decode_q8_kernel<D, FMT, NT, kWeights>, static_cast<int>(sizeof(Shared<D, NT>)), smem_set))
        return -1;
    constexpr int W = warps_of(NT);
    if (blocks <= W) return 1;
    int64_t cl = (blocks + W - 1) / W;
    if (cl > kMaxCluster) cl = kMaxCluster;
    if (cl > num_sms() / heads) cl = num_sms() / heads;
    while (cl > 1 && heads > max_clusters<D, FMT, NT, kWeights>(static_cast<int>(cl))) --cl;
    if (cl < 1) cl = 1;
    const int64_t units = (blocks + W * cl - 1) / (W * cl);  // of a warp
    if (units > (cl == 1 ? 2 : 4)) return 0;
    return static_cast<int>((blocks + W * units - 1) / (W * units));
}

template <int D, int FMT, int NT, bool kWeights>
static tg_status launch(DecodeArgs& a, int64_t blocks, cudaStream_t st) {
    const int64_t heads = static_cast<int64_t>(a.c.batch) * a.c.Hkv;
    a.cluster = cluster_for<D, FMT, NT, kWeights>(heads, blocks);
    if (a.cluster < 0) return TG_ERR_CUDA;
    const int64_t sms = num_sms() < kMaxParts ? num_sms() : kMaxParts, grid = a.cluster ? heads * a.cluster : sms;
    auto kern = gated_decode_q8_kernel<D, FMT, NT, kWeights>;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(static_cast<unsigned>(grid));
    cfg.blockDim = dim3(warps_of(NT) * 32);
    cfg.dynamicSmemBytes = sizeof(Shared<D, NT>);
    cfg.stream = st;
    cudaLaunchAttribute at[2] = {pdl_attr()};
    at[1].id = cudaLaunchAttributeClusterDimension;
    at[1].val.clusterDim.x = static_cast<unsigned>(a.cluster);
    at[1].val.clusterDim.y = at[1].val.clusterDim.z = 1;
    cfg.attrs = at;
    cfg.numAttrs = a.cluster > 1 ? 2 : 1;
    return cudaLaunchKernelEx(&cfg, kern, a) == cudaSuccess ? launch_status() : TG_ERR_CUDA;
}

template <int D, int FMT>
static tg_status launch_rows(DecodeArgs& a, bool weights, int64_t blocks, cudaStream_t st) {
    if (a.R <= 8) return weights ? launch<D, FMT, 1, true>(a, blocks, st) : launch<D, FMT, 1, false>(a, blocks, st);
    return weights ? launch<D, FMT, 2, true>(a, blocks, st) : launch<D, FMT, 2, false>(a, blocks, st);
}

}  // namespace q8
}  // namespace tg

using namespace tg;

extern "C" size_t tg_cache_workspace_bytes(const tg_cache_q8* cache, int32_t n_q, int32_t Hq, int32_t accumulate) {
    q8::Cache c;
    if (!cache || n_q < 0 || Hq < 0) return 0;
    tg_cache_q8 shape = *cache;          // the sizes alone count here
    shape.k = shape.v = reinterpret_cast<void*>(16);
    shape.k_scale = shape.v_scale = reinterpret_cast<float*>(16);
    shape.lengths = reinterpret_cast<int32_t*>(16);
    if (q8::check_cache(&shape, &c) != TG_OK) return 0;
    if (n_q == 0 || Hq == 0) return kWsHeader;
    if (Hq % c.Hkv || static_cast<int64_t>(n_q) * (Hq / c.Hkv) > q8::kMaxRows) return 0;
    return q8::layout(c, shape.d_h, n_q * (Hq / c.Hkv), accumulate != 0).bytes;
}

extern "C" tg_status tg_gated_decode_q8(const tg_cache_q8* cache, const tg_bf16* q, int32_t n_q, int32_t Hq,
                                        const float* gain, float tau, int32_t accumulate, int64_t max_len,
                                        tg_bf16* out, float* lse, void* workspace, size_t workspace_bytes,
                                        void* stream) {
    q8::DecodeArgs a = {};
    const tg_status ok = q8::check_cache(cache, &a.c);
    if (ok != TG_OK) return ok;
    if (n_q <= 0 || Hq <= 0 || Hq % a.c.Hkv || !std::isfinite(tau) || max_len < 0) return TG_ERR_INVALID_ARG;
    if (accumulate && a.c.capacity > 0 && !a.c.w) return TG_ERR_INVALID_ARG;
    a.G = Hq / a.c.Hkv;
    if (static_cast<int64_t>(n_q) * a.G > q8::kMaxRows) return TG_ERR_UNSUPPORTED;
    if (a.c.batch == 0) return TG_OK;
    if (!q || !out || !workspace || !aligned16(q) || !aligned16(out) || !aligned16(workspace))
        return TG_ERR_INVALID_ARG;
    // the queries are read while finished rows are written
    const size_t row_bytes = static_cast<size_t>(a.c.batch) * n_q * Hq * cache->d_h * sizeof(tg_bf16);
    if (q8::overlap(q, row_bytes, out, row_bytes)) return TG_ERR_INVALID_ARG;
    a.R = n_q * a.G;
    a.Rp = (a.R + 1) / 2 * 2;
    const q8::Layout L = q8::layout(a.c, cache->d_h, a.R, accumulate != 0);
    if (workspace_bytes < L.bytes) return TG_ERR_INVALID_ARG;
    char* ws = static_cast<char*>(workspace);
    a.q = reinterpret_cast<const __nv_bfloat16*>(q);
    a.gain = gain;
    a.out = reinterpret_cast<__nv_bfloat16*>(out);
    a.lse = lse;
    a.scale = tau / std::sqrt(static_cast<float>(cache->d_h));
    a.n_q = n_q;
    a.Hq = Hq;
    a.status = status_word(workspace);
    a.heads = reinterpret_cast<int2*>(ws + L.heads);
    a.rows = reinterpret_cast<float2*>(ws + L.rows);
    a.part = reinterpret_cast<float*>(ws + L.part);
    a.part_ml = reinterpret_cast<float2*>(ws + L.part_ml);
    a.logits = reinterpret_cast<float*>(ws + L.logits);
    if (max_len == 0 || max_len > a.c.capacity) max_len = a.c.capacity;
    const int64_t blocks = (max_len + q8::kBlock - 1) / q8::kBlock;
    cudaStream_t st = as_stream(stream);
    const bool w = accumulate != 0 && a.c.capacity > 0;
    tg_status r;
    if (cache->d_h == 128)
        r = cache->format == TG_CACHE_E4M3 ? q8::launch_rows<128, TG_CACHE_E4M3>(a, w, blocks, st)
                                           : q8::launch_rows<128, TG_CACHE_INT8>(a, w, blocks, st);
    else
        r = cache->format == TG_CACHE_E4M3 ? q8::launch_rows<64, TG_CACHE_E4M3>(a, w, blocks, st)
                                           : q8::launch_rows<64, TG_CACHE_INT8>(a, w, blocks, st);
    if (r != TG_OK || (a.cluster && !w)) return r;
    int64_t x = w ? (max_len + q8::kWeightKeys - 1) / q8::kWeightKeys : 0;
    if (x > 4 * num_sms() / a.c.batch) x = 4 * num_sms() / a.c.batch;   // one wave (the rest by the kernel's stride)
    if (w && x < 1) x = 1;
    const int rows = q8::kMergeVecs / (cache->d_h / 4);
    const int merges = a.cluster ? 0 : a.c.Hkv * ((a.R + rows - 1) / rows);
    const dim3 fin(static_cast<unsigned>(merges + x), static_cast<unsigned>(a.c.batch));
    return q8::launch_pdl(cache->d_h == 128 ? q8::decode_q8_finish_kernel<128> : q8::decode_q8_finish_kernel<64>, fin,
                          dim3(q8::kFinThreads), 0, st, a, merges);
}
