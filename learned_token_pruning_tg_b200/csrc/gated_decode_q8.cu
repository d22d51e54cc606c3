// gated_decode_q8.cu -- decoding steps of token-gated attention over an 8-bit KV cache.
//
// With codes K, V and one scale per block of 32 keys and head, for the R = n_q G query
// rows that read one KV head:
//   x_rc = (tau / sqrt(d) log2 e) kscale (q_r . K_c) + g_r s_c log2 e      (log2 units)
//   out_r = sum_blocks vscale sum_{c in block} 2^(x_rc - m_r) V_c / sum_c 2^(x_rc - m_r)
// The cache is read once: 2 d bytes a key and head, so HBM bounds a long step and latency a
// short one.
//
// Work: a unit is one block (32 keys) of one head of one sequence.  The units of all
// sequences, in order (sequence, head, block), are cut into equal runs, one for every thread block
// of the launch (counted on the device from `lengths`, so one captured launch serves
// growing and ragged sequences evenly); the warps of a thread block take the units of a run in
// turn.  Each warp keeps its own running max, sum and output; they merge in shared memory when
// a head's run ends, and a head that several thread blocks share is merged by the last of them to
// arrive (a counter in the workspace), in the order of the runs, so results do not depend on timing.
//
// A unit in a warp: K and V codes come straight from global memory into registers in the layout
// of mma.m16n8k16's A operand -- keys (K) or head dimensions (V, transposed by byte
// permutes) as the 16 rows, the query rows as the 8 columns of B: few queries waste
// columns of a small MMA, not rows of a large one.  The order of d inside a dot product and of
// the output's d over MMA rows is free, so every lane reads 16 contiguous bytes at a time and no
// shared memory is involved.  S^T = K Q^T leaves weights whose 8x8 pieces movmatrix turns into the
// B operand of O^T += V^T P^T.  Codes are exact in fp16.  The next unit's K is on its way
// while this one's softmax and V product run, and the next V behind them.  (tcgen05 would take 128
// keys a step from shared memory and bring the 8 columns back through TMEM; the products are far from
// the bound here.)
//
// Roundings: q is scaled to fp16 by a power of two per row (bf16 has fewer bits: only
// elements 2^-25 of the row's largest are lost); the weights 2^(x - m + 15) are rounded to fp16 for
// the V product (2^-12 each, below the output's bf16; the 15 keeps weights down to 2^-29 of the
// largest normal), their sum is not.
#include <cmath>

#include "tg_cache.cuh"

namespace tg {
namespace q8 {

constexpr int kWarps = 4;
constexpr int kMaxRows = 16;             // query rows per KV head
constexpr int kMaxCtas = 148 * 8;
constexpr int kMaxShare = 256;           // thread blocks that share one head at most (on average)
constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;
constexpr float kShift = 15.0f;          // weights are 2^(x - m + kShift)
constexpr int kWeightThreads = 256;

struct DecodeArgs {
    Cache c;
    const __nv_bfloat16* q;
    const float* gain;
    __nv_bfloat16* out;
    float* lse;
    float scale_log2;                    // tau / sqrt(d) * log2(e)
    int n_q, Hq, G, R;
    int Rp;                              // R rounded up to even: a key's logits in the workspace
    unsigned int* status;
    unsigned int* counter;               // [batch * Hkv], zero between calls
    float* lse2;                         // [batch * Hkv][kMaxRows], log2 units
    float* part;                         // [2 * grid][R][2 + d]: m, l, o of a run's first / last head
    float* logits;                       // [batch * Hkv][capacity][Rp] log2 units
};

__device__ __forceinline__ float ex2(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

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

// Sum over the block of one value per thread (every thread gets it).
__device__ __forceinline__ long long block_sum(long long v, long long* s_warp) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
    if ((threadIdx.x & 31) == 0) s_warp[threadIdx.x >> 5] = v;
    __syncthreads();
    long long t = 0;
#pragma unroll
    for (int w = 0; w < kWarps; ++w) t += s_warp[w];
    __syncthreads();
    return t;
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
    float f[NT][2], gl2[NT][2];          // logit factor and gain of this lane's query rows 8 nt + 2 t + {0, 1}
    int cut[NT][2];                      // keys those rows do not see at the sequence's end
    float m[NT][2], l[NT][2], o[D / 16][NT][4];

    __device__ __forceinline__ explicit Warp(const DecodeArgs& args)
        : a(args), lane(threadIdx.x & 31), g(lane >> 2), t(lane & 3) {}

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
            e = e > 127 ? 0 : max(e, -126);
            const float down = __int_as_float((127 - min(e, 126)) << 23);
            const float up = __fdiv_rn(1.0f, down);
#pragma unroll
            for (int j = 0; j < D / 16; ++j) {
                const float* y = &x[j / 4][4 * (j % 4)];
                qf[j][nt][0] = pack_f16x2(y[0] * down, y[1] * down);
                qf[j][nt][1] = pack_f16x2(y[2] * down, y[3] * down);
            }
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                f[nt][i] = __shfl_sync(0xffffffffu, up, 4 * (2 * t + i)) * a.scale_log2;
                const int rr = 8 * nt + 2 * t + i;
                gl2[nt][i] = (rr < a.R && a.gain) ? __ldg(a.gain + kvh * a.G + rr % a.G) * kLog2e : 0.0f;
                cut[nt][i] = rr < a.R ? a.n_q - 1 - rr / a.G : 0;
                m[nt][i] = -INFINITY;
                l[nt][i] = 0.0f;
            }
        }
#pragma unroll
        for (int dm = 0; dm < D / 16; ++dm)
#pragma unroll
            for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                for (int i = 0; i < 4; ++i) o[dm][nt][i] = 0.0f;
    }

    __device__ __forceinline__ void load_keys(KeyRegs<D>& k, int b, int kvh, int blk) const {
        const uint8_t* base = a.c.k + b * a.c.ld_seq + static_cast<int64_t>(blk) * kBlock * a.c.ld_token + kvh * D;
#pragma unroll
        for (int r = 0; r < 4; ++r)
#pragma unroll
            for (int i = 0; i < D / 64; ++i)
                load_codes<4>(base + (8 * r + g) * a.c.ld_token + 64 * i + 16 * t, &k.w[r][4 * i]);
        k.scale = __ldg(a.c.k_scale + (b * a.c.blocks() + blk) * a.c.Hkv + kvh);
        if (a.c.s) {
#pragma unroll
            for (int r = 0; r < 4; ++r) k.s[r] = __ldg(a.c.s + b * a.c.capacity + blk * kBlock + 8 * r + g);
        }
    }
    __device__ __forceinline__ void load_values(ValueRegs<D>& v, int b, int kvh, int blk) const {
        const uint8_t* base = a.c.v + b * a.c.ld_seq + static_cast<int64_t>(blk) * kBlock * a.c.ld_token + kvh * D;
#pragma unroll
        for (int i = 0; i < 2; ++i)
#pragma unroll
            for (int j = 0; j < 4; ++j)
                load_codes<D / 32>(base + (16 * i + 2 * t + (j & 1) + 8 * (j >> 1)) * a.c.ld_token + g * (D / 8),
                                   v.w[i][j]);
        v.scale = __ldg(a.c.v_scale + (b * a.c.blocks() + blk) * a.c.Hkv + kvh);
    }

    // Logits of a unit, the weights as B operands, the running max and sum; alpha: by how much
    // the sums before shrink.
    __device__ __forceinline__ void scores(const KeyRegs<D>& k, int b, int kvh, int blk, int len,
                                           uint32_t (&pf)[2][NT][2], float (&alpha)[NT][2]) {
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
        const bool ragged = (blk + 1) * kBlock > len - (a.n_q - 1);
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
            float mx[2] = {-INFINITY, -INFINITY};
#pragma unroll
            for (int i = 0; i < 2; ++i)
#pragma unroll
                for (int c = 0; c < 4; ++c) {
                    float y = x[i][nt][c] * (f[nt][c & 1] * k.scale);
                    if (bias) y = fmaf(gl2[nt][c & 1], k.s[2 * i + (c >> 1)], y);
                    if (ragged && blk * kBlock + 16 * i + 8 * (c >> 1) + g >= len - cut[nt][c & 1]) y = -INFINITY;
                    x[i][nt][c] = y;
                    mx[c & 1] = fmaxf(mx[c & 1], y);
                }
            if constexpr (kWeights) {
                if (8 * nt + 2 * t < a.R) {
                    float* to = a.logits +
                                ((static_cast<int64_t>(b) * a.c.Hkv + kvh) * a.c.capacity + blk * kBlock + g) * a.Rp +
                                8 * nt + 2 * t;
#pragma unroll
                    for (int r = 0; r < 4; ++r)
                        *reinterpret_cast<float2*>(to + 8 * r * a.Rp) =
                            make_float2(x[r >> 1][nt][2 * (r & 1)], x[r >> 1][nt][2 * (r & 1) + 1]);
                }
            }
#pragma unroll
            for (int c = 0; c < 2; ++c) {
#pragma unroll
                for (int off = 4; off < 32; off <<= 1) mx[c] = fmaxf(mx[c], __shfl_xor_sync(0xffffffffu, mx[c], off));
                const float mn = fmaxf(m[nt][c], mx[c]);
                const float base = mn == -INFINITY ? 0.0f : mn;      // nothing seen yet: every weight is 0
                alpha[nt][c] = ex2(m[nt][c] - base);
                m[nt][c] = mn;
                l[nt][c] *= alpha[nt][c];
                mx[c] = base - kShift;
            }
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                float p[4];
#pragma unroll
                for (int c = 0; c < 4; ++c) {
                    p[c] = ex2(x[i][nt][c] - mx[c & 1]);
                    l[nt][c & 1] += p[c];
                }
                pf[i][nt][0] = transpose8x8(pack_f16x2(p[0], p[1]));
                pf[i][nt][1] = transpose8x8(pack_f16x2(p[2], p[3]));
            }
        }
    }

    __device__ __forceinline__ void values(ValueRegs<D>& v, int blk, int len, const uint32_t (&pf)[2][NT][2],
                                           const float (&alpha)[NT][2]) {
        if ((blk + 1) * kBlock > len) {
            // rows behind the sequence may hold anything, NaN codes too: their weight is 0
#pragma unroll
            for (int i = 0; i < 2; ++i)
#pragma unroll
                for (int j = 0; j < 4; ++j)
                    if (blk * kBlock + 16 * i + 2 * t + (j & 1) + 8 * (j >> 1) >= len)
#pragma unroll
                        for (int w = 0; w < D / 32; ++w) v.w[i][j][w] = 0u;
        }
#pragma unroll
        for (int dm = 0; dm < D / 16; ++dm) {
            float acc[NT][4];
#pragma unroll
            for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                for (int c = 0; c < 4; ++c) acc[nt][c] = 0.0f;
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
#pragma unroll
            for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                for (int c = 0; c < 4; ++c)
                    o[dm][nt][c] = fmaf(v.scale, acc[nt][c], o[dm][nt][c] * alpha[nt][c & 1]);
        }
    }

    // Units u0 + warp, u0 + warp + kWarps, ... < u1 of one head.
    __device__ __forceinline__ void run(int b, int kvh, int u0, int u1, int len) {
        begin(b, kvh);
        int u = u0 + (threadIdx.x >> 5);
        KeyRegs<D> k;
        ValueRegs<D> v;
        if (u < u1) {
            load_keys(k, b, kvh, u);
            load_values(v, b, kvh, u);
        }
        for (; u < u1; u += kWarps) {
            uint32_t pf[2][NT][2];
            float alpha[NT][2];
            const int next = u + kWarps;
            scores(k, b, kvh, u, len, pf, alpha);
            if (next < u1) load_keys(k, b, kvh, next);
            values(v, u, len, pf, alpha);
            if (next < u1) load_values(v, b, kvh, next);
        }
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int c = 0; c < 2; ++c)
#pragma unroll
                for (int off = 4; off < 32; off <<= 1) l[nt][c] += __shfl_xor_sync(0xffffffffu, l[nt][c], off);
    }
};

// One row's answer from its sums (weights carry 2^kShift).
__device__ __forceinline__ void finish_row(const DecodeArgs& a, int b, int kvh, int r, float m, float l) {
    const float lse2 = l == 0.0f ? -INFINITY : m + log2f(l) - kShift;
    a.lse2[(static_cast<int64_t>(b) * a.c.Hkv + kvh) * kMaxRows + r] = lse2;
    if (a.lse) a.lse[(static_cast<int64_t>(b) * a.n_q + r / a.G) * a.Hq + kvh * a.G + r % a.G] = lse2 * kLn2;
}
__device__ __forceinline__ __nv_bfloat16* out_row(const DecodeArgs& a, int b, int kvh, int r, int D) {
    return a.out + ((static_cast<int64_t>(b) * a.n_q + r / a.G) * a.Hq + kvh * a.G + r % a.G) * D;
}

template <int D, int FMT, int NT, bool kWeights>
__global__ void __launch_bounds__(kWarps * 32, NT == 1 ? 3 : 2) gated_decode_q8_kernel(const DecodeArgs a) {
    __shared__ float s_m[kWarps][8 * NT], s_l[kWarps][8 * NT];
    __shared__ __align__(16) float s_o[kWarps * 8 * NT * D];
    __shared__ long long s_red[kWarps];
    __shared__ int s_b;
    __shared__ long long s_base;
    __shared__ bool s_last;
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    pdl_wait();
    pdl_trigger();
    const int B = a.c.batch, Hkv = a.c.Hkv;
    const int64_t G_all = gridDim.x;

    // sequences without a token have no units: their rows are 0
    for (int b = blockIdx.x; b < B; b += gridDim.x) {
        if (length_of(a.c, b, a.status) > 0) continue;
        for (int i = tid; i < a.n_q * a.Hq * D; i += kWarps * 32)
            a.out[static_cast<int64_t>(b) * a.n_q * a.Hq * D + i] = __float2bfloat16_rn(0.0f);
        for (int i = tid; i < Hkv * a.R; i += kWarps * 32) finish_row(a, b, i / a.R, i % a.R, 0.0f, 0.0f);
    }

    // this thread block's run of units, and the sequence in which it begins
    auto units_of = [&](int b) -> long long {
        return static_cast<long long>((length_of(a.c, b, a.status) + kBlock - 1) / kBlock) * Hkv;
    };
    long long total = 0;
    if (B == 1) {
        total = units_of(0);
    } else {
        for (int b = tid; b < B; b += kWarps * 32) total += units_of(b);
        total = block_sum(total, s_red);
    }
    const long long n = G_all < total ? G_all : total;
    if (blockIdx.x >= n) return;
    long long u = total * blockIdx.x / n;
    const long long u_end = total * (blockIdx.x + 1) / n;
    const long long u_begin = u;
    int b = 0;
    long long base = 0;                   // units before sequence b
    if (B > 1) {
        for (int b0 = 0;; b0 += kWarps * 32) {
            const long long mine = b0 + tid < B ? units_of(b0 + tid) : 0;
            long long incl = mine;
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const long long y = __shfl_up_sync(0xffffffffu, incl, o);
                if (lane >= o) incl += y;
            }
            if (lane == 31) s_red[warp] = incl;
            __syncthreads();
            long long before = base;
            for (int w = 0; w < warp; ++w) before += s_red[w];
            long long all = base;
            for (int w = 0; w < kWarps; ++w) all += s_red[w];
            if (before + incl - mine <= u && u < before + incl) {
                s_b = b0 + tid;
                s_base = before + incl - mine;
            }
            __syncthreads();
            if (u < all) break;
            base = all;
        }
        b = s_b;
        base = s_base;
    }

    Warp<D, FMT, NT, kWeights> wp(a);
    while (u < u_end) {
        const int len = length_of(a.c, b, a.status);
        const int nblk = (len + kBlock - 1) / kBlock;
        if (nblk == 0) {                  // nothing here: the next sequence
            ++b;
            continue;
        }
        const int kvh = static_cast<int>((u - base) / nblk);
        const long long seg = base + static_cast<long long>(kvh) * nblk;
        const long long stop = seg + nblk < u_end ? seg + nblk : u_end;
        wp.run(b, kvh, static_cast<int>(u - seg), static_cast<int>(stop - seg), len);

        // the warps' sums of this head
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
            if (wp.g == 0) {
#pragma unroll
                for (int c = 0; c < 2; ++c) {
                    s_m[warp][8 * nt + 2 * wp.t + c] = wp.m[nt][c];
                    s_l[warp][8 * nt + 2 * wp.t + c] = wp.l[nt][c];
                }
            }
#pragma unroll
            for (int c = 0; c < 2; ++c) {
                const int r = 8 * nt + 2 * wp.t + c;
                if (r < a.R) {
                    float* to = s_o + (warp * 8 * NT + r) * D + D / 8 * wp.g;
#pragma unroll
                    for (int dm = 0; dm < D / 16; ++dm)
                        *reinterpret_cast<float2*>(to + 2 * dm) =
                            make_float2(wp.o[dm][nt][c], wp.o[dm][nt][2 + c]);
                }
            }
        }
        __syncthreads();
        // thread blocks that share this head: those holding its first and last unit, and all between
        const long long i0 = ((seg + 1) * n - 1) / total, i1 = ((seg + nblk) * n - 1) / total;
        const bool whole = i0 == i1;
        float* part = a.part + (2 * blockIdx.x + (seg < u_begin ? 0 : 1)) * static_cast<int64_t>(a.R) * (2 + D);
        for (int i = tid; i < a.R * D; i += kWarps * 32) {
            const int r = i / D, d = i % D;
            float mx = -INFINITY;
#pragma unroll
            for (int w = 0; w < kWarps; ++w) mx = fmaxf(mx, s_m[w][r]);
            const float ref = mx == -INFINITY ? 0.0f : mx;
            float ls = 0.0f, os = 0.0f;
#pragma unroll
            for (int w = 0; w < kWarps; ++w) {
                const float fw = ex2(s_m[w][r] - ref);
                ls += s_l[w][r] * fw;
                os += s_o[(w * 8 * NT + r) * D + d] * fw;
            }
            if (whole) {
                out_row(a, b, kvh, r, D)[d] = __float2bfloat16_rn(ls == 0.0f ? 0.0f : os / ls);
                if (d == 0) finish_row(a, b, kvh, r, ref, ls);
            } else {
                part[r * (2 + D) + 2 + d] = os;
                if (d == 0) {
                    part[r * (2 + D)] = mx;
                    part[r * (2 + D) + 1] = ls;
                }
            }
        }
        if (!whole) {
            __threadfence();
            __syncthreads();
            unsigned int* count = a.counter + static_cast<int64_t>(b) * Hkv + kvh;
            if (tid == 0) s_last = atomicAdd(count, 1u) == static_cast<unsigned>(i1 - i0);
            __syncthreads();
            if (s_last) {
                __threadfence();
                const int np = static_cast<int>(i1 - i0) + 1;
                // part p belongs to thread block i0 + p: its last head for p = 0, its first one otherwise
                const float* parts = a.part;
                const int64_t ld = static_cast<int64_t>(a.R) * (2 + D);
                for (int i = tid; i < a.R * D; i += kWarps * 32) {
                    const int r = i / D, d = i % D;
                    float mx = -INFINITY;
                    for (int p = 0; p < np; ++p)
                        mx = fmaxf(mx, __ldcg(parts + (2 * (i0 + p) + (p == 0)) * ld + r * (2 + D)));
                    const float ref = mx == -INFINITY ? 0.0f : mx;
                    float ls = 0.0f, os = 0.0f;
                    for (int p = 0; p < np; ++p) {
                        const float* pr = parts + (2 * (i0 + p) + (p == 0)) * ld + r * (2 + D);
                        const float fp = ex2(__ldcg(pr) - ref);
                        ls += __ldcg(pr + 1) * fp;
                        os += __ldcg(pr + 2 + d) * fp;
                    }
                    out_row(a, b, kvh, r, D)[d] = __float2bfloat16_rn(ls == 0.0f ? 0.0f : os / ls);
                    if (d == 0) finish_row(a, b, kvh, r, ref, ls);
                }
                if (tid == 0) *count = 0u;   // ready for the next call
            }
        }
        __syncthreads();                  // the shared sums are free again
        u = stop;
        if (u == seg + nblk && kvh == Hkv - 1) {
            base += static_cast<long long>(nblk) * Hkv;
            ++b;
        }
    }
}

// w[b, c] += sum over the heads' rows of 2^(x - lse2): one thread a key, a fixed order.
__global__ void __launch_bounds__(kWeightThreads) decode_q8_weights_kernel(const DecodeArgs a) {
    __shared__ float s_lse[64 * kMaxRows];
    pdl_wait();
    pdl_trigger();
    const int b = blockIdx.y, len = length_of(a.c, b, a.status);
    for (int i = threadIdx.x; i < a.c.Hkv * a.Rp; i += kWeightThreads) {
        const int h = i / a.Rp, r = i % a.Rp;
        const float v = r < a.R ? a.lse2[(static_cast<int64_t>(b) * a.c.Hkv + h) * kMaxRows + r] : INFINITY;
        s_lse[i] = v == -INFINITY ? INFINITY : v;   // a row that saw nothing adds nothing
    }
    __syncthreads();
    for (int64_t c = static_cast<int64_t>(blockIdx.x) * kWeightThreads + threadIdx.x; c < len;
         c += static_cast<int64_t>(gridDim.x) * kWeightThreads) {
        float sum = 0.0f;
        for (int h = 0; h < a.c.Hkv; ++h) {
            const float* x = a.logits + ((static_cast<int64_t>(b) * a.c.Hkv + h) * a.c.capacity + c) * a.Rp;
            for (int r = 0; r < a.Rp; r += 2) {
                const float2 y = __ldcg(reinterpret_cast<const float2*>(x + r));
                sum += ex2(y.x - s_lse[h * a.Rp + r]);
                if (r + 1 < a.R) sum += ex2(y.y - s_lse[h * a.Rp + r + 1]);
            }
        }
        a.c.w[b * a.c.capacity + c] += sum;
    }
}

// Workspace: status header, counters, lse2, parts, logits (each from a 256-byte boundary).
struct Layout {
    size_t counter, lse2, part, logits, bytes;
};
static size_t up256(size_t x) { return (x + 255) / 256 * 256; }
static int max_grid(int64_t heads) {
    return static_cast<int>(heads * kMaxShare < kMaxCtas ? heads * kMaxShare : kMaxCtas);
}
static Layout layout(const Cache& c, int d_h, int R, bool weights) {
    const int64_t heads = static_cast<int64_t>(c.batch) * c.Hkv;
    Layout L;
    L.counter = kWsHeader;
    L.lse2 = L.counter + up256(static_cast<size_t>(heads) * 4);
    L.part = L.lse2 + up256(static_cast<size_t>(heads) * kMaxRows * 4);
    L.logits = L.part + up256(static_cast<size_t>(max_grid(heads)) * 2 * R * (2 + d_h) * 4);
    L.bytes = L.logits + (weights ? up256(static_cast<size_t>(heads) * c.capacity * ((R + 1) / 2 * 2) * 4) : 0);
    return L;
}

template <int D, int FMT, int NT, bool kWeights>
static tg_status launch(const DecodeArgs& a, int64_t max_units, cudaStream_t st) {
    static std::atomic<int> occ_cache[64];
    const int dev = current_device();
    auto kern = gated_decode_q8_kernel<D, FMT, NT, kWeights>;
    int occ = dev >= 0 ? occ_cache[dev].load(std::memory_order_relaxed) : 0;
    if (occ <= 0) {
        if (cudaOccupancyMaxActiveBlocksPerMultiprocessor(&occ, kern, kWarps * 32, 0) != cudaSuccess || occ <= 0) occ = 1;
        if (dev >= 0) occ_cache[dev].store(occ, std::memory_order_relaxed);
    }
    // one wave of resident thread blocks, a unit for every warp
    int64_t grid = static_cast<int64_t>(num_sms()) * occ;
    const int64_t most = max_grid(static_cast<int64_t>(a.c.batch) * a.c.Hkv);
    if (grid > most) grid = most;
    if (grid > (max_units + kWarps - 1) / kWarps) grid = (max_units + kWarps - 1) / kWarps;
    if (grid < 1) grid = 1;
    return launch_pdl(kern, dim3(static_cast<unsigned>(grid)), dim3(kWarps * 32), 0, st, a);
}

template <int D, int FMT>
static tg_status launch_rows(const DecodeArgs& a, bool weights, int64_t max_units, cudaStream_t st) {
    if (a.R <= 8)
        return weights ? launch<D, FMT, 1, true>(a, max_units, st) : launch<D, FMT, 1, false>(a, max_units, st);
    return weights ? launch<D, FMT, 2, true>(a, max_units, st) : launch<D, FMT, 2, false>(a, max_units, st);
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
    a.R = n_q * a.G;
    a.Rp = (a.R + 1) / 2 * 2;
    const q8::Layout L = q8::layout(a.c, cache->d_h, a.R, accumulate != 0);
    if (workspace_bytes < L.bytes) return TG_ERR_INVALID_ARG;
    char* ws = static_cast<char*>(workspace);
    a.q = reinterpret_cast<const __nv_bfloat16*>(q);
    a.gain = gain;
    a.out = reinterpret_cast<__nv_bfloat16*>(out);
    a.lse = lse;
    a.scale_log2 = tau / std::sqrt(static_cast<float>(cache->d_h)) * q8::kLog2e;
    a.n_q = n_q;
    a.Hq = Hq;
    a.status = status_word(workspace);
    a.counter = reinterpret_cast<unsigned int*>(ws + L.counter);
    a.lse2 = reinterpret_cast<float*>(ws + L.lse2);
    a.part = reinterpret_cast<float*>(ws + L.part);
    a.logits = reinterpret_cast<float*>(ws + L.logits);
    if (max_len == 0 || max_len > a.c.capacity) max_len = a.c.capacity;
    const int64_t max_units = (max_len + q8::kBlock - 1) / q8::kBlock * a.c.Hkv * a.c.batch;
    cudaStream_t st = as_stream(stream);
    const bool w = accumulate != 0 && a.c.capacity > 0;
    tg_status r;
    if (cache->d_h == 128)
        r = cache->format == TG_CACHE_E4M3 ? q8::launch_rows<128, TG_CACHE_E4M3>(a, w, max_units, st)
                                           : q8::launch_rows<128, TG_CACHE_INT8>(a, w, max_units, st);
    else
        r = cache->format == TG_CACHE_E4M3 ? q8::launch_rows<64, TG_CACHE_E4M3>(a, w, max_units, st)
                                           : q8::launch_rows<64, TG_CACHE_INT8>(a, w, max_units, st);
    if (r != TG_OK || !w) return r;
    int64_t blocks = (max_len + q8::kWeightThreads - 1) / q8::kWeightThreads;
    if (blocks > 4096) blocks = 4096;
    return q8::launch_pdl(q8::decode_q8_weights_kernel,
                          dim3(static_cast<unsigned>(blocks < 1 ? 1 : blocks), static_cast<unsigned>(a.c.batch)),
                          dim3(q8::kWeightThreads), 0, st, a);
}
