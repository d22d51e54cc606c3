// cache_q8.cu -- the 8-bit KV cache's own calls: append, read back, evict.
//
// A block is 32 tokens of one head (K and V apart) under one scale 2^e, the least with amax <= qmax 2^e.
// Every kernel here moves bytes: one warp holds one block in registers, so the largest magnitude is a
// warp reduction and the block is read and written once.
//
// append: bf16 rows (2 rows a warp load, 16 bytes a lane) -> codes (8 bytes a lane).  A block with tokens of an
//   earlier append keeps the larger scale; its codes move to it by one multiplication with a power
//   of two and one rounding.  HBM bounds a prompt: 65536 tokens of 8 heads of 128 (403 MB) take 63.5 us, 6.4 TB/s
//   (replayed in a graph; 67 us as calls one by one); one token is a launch (2.6 us in a graph).
// evict: one thread block, or a cluster of them, finds a sequence's kept slots by a radix select over the
//   weights (11 + 11 + 10 bits of the order-preserving key), then one warp per new block gathers its 32 rows.
//   Latency bounds both: 8961 tokens to 8704 (36 MB) 20.4 us, 65537 to 8704 23.3 us, half of either the select.
//   (4 rows, or 1, a lane instead of 8: 1.0 and 1.8 us more.)
// read: HBM or L2 bounds it (24 MB of ragged sequences in about 6 us).
#include "tg_cache.cuh"

namespace tg {
namespace q8 {

constexpr int kWarps = 4;                // warps of an append or gather thread block (8: 67.5 us for the prompt below)
constexpr int kReadThreads = 256;
constexpr float kMostRatio = 262144.0f;  // 2^18 > 448 / 2^-9, the largest and the least code of e4m3 (int8: 128)

__device__ __forceinline__ float warp_max(float v) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, o));
    return v;
}

// ------------------------------------------------------------------------------------------- append
struct AppendArgs {
    Cache c;
    const __nv_bfloat16 *k, *v;
    int64_t ld_k, ld_k_seq, ld_v, ld_v_seq;
    int64_t n_new;
    const int32_t* counts;
    const float* s_new;
    unsigned int* status;
    int units;                           // blocks a sequence's new tokens may touch * Hkv * 2
};

// One warp: block j of one head of K or V.  Rows [first, last) of the block are new (their tokens start at
// `x`), rows before them stay.
template <int D, int FMT>
__device__ __forceinline__ void append_block(const __nv_bfloat16* x, int64_t ld, uint8_t* codes, int64_t ld_token,
                                             float* scale, int first, int last, unsigned int* status) {
    constexpr int LPR = D / 8;           // lanes of a row (8 elements, 16 bytes each)
    constexpr int RPL = 32 / LPR;        // rows a warp load covers
    constexpr int N = kBlock / RPL;
    const int lane = threadIdx.x & 31, row0 = lane / LPR, col = (lane % LPR) * 8;
    uint4 u[N];
    uint32_t top = 0;                    // the largest magnitudes, as bf16 bits in either half
#pragma unroll
    for (int i = 0; i < N; ++i) {
        const int r = i * RPL + row0;
        u[i] = (r >= first && r < last) ? __ldg(reinterpret_cast<const uint4*>(x + (r - first) * ld + col))
                                        : make_uint4(0u, 0u, 0u, 0u);
    }
#pragma unroll
    for (int i = 0; i < N; ++i) {
        top = __vmaxu2(top, u[i].x & 0x7fff7fffu);
        top = __vmaxu2(top, u[i].y & 0x7fff7fffu);
        top = __vmaxu2(top, u[i].z & 0x7fff7fffu);
        top = __vmaxu2(top, u[i].w & 0x7fff7fffu);
    }
    uint32_t bits = max(top & 0xffffu, top >> 16);
    bits = __reduce_max_sync(0xffffffffu, bits);
    const bool odd = bits >= 0x7f80u;    // an infinity or a NaN: the largest finite magnitude instead
    if (odd) {
        bits = 0;
#pragma unroll
        for (int i = 0; i < N; ++i) {
            const uint32_t w[4] = {u[i].x, u[i].y, u[i].z, u[i].w};
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const uint32_t lo = w[j] & 0x7fffu, hi = (w[j] >> 16) & 0x7fffu;
                if (lo < 0x7f80u) bits = max(bits, lo);
                if (hi < 0x7f80u) bits = max(bits, hi);
            }
        }
        bits = __reduce_max_sync(0xffffffffu, bits);
        if (lane == 0) atomicOr(status, TG_STATUS_CACHE_VALUE);
    }
    float sc = scale_for<FMT>(__uint_as_float(bits << 16));
    if (first > 0) {
        const float before = *scale;
        if (before >= sc) {
            sc = before;
        } else if (before > 0.0f) {      // (codes without a scale that is a number stand for nothing: they stay)
            // the scale grows: the block's earlier codes once more
            const float ratio = __fdiv_rn(before, sc);
            constexpr int LPC = D / 16;  // lanes of a row of codes (16 bytes each)
            for (int r = lane / LPC; r < first; r += 32 / LPC) {
                uint4* p = reinterpret_cast<uint4*>(codes + r * ld_token + (lane % LPC) * 16);
                const uint4 c = *p;
                uint32_t w[4] = {c.x, c.y, c.z, c.w};
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    float f[4];
                    decode4<FMT>(w[j], f);
                    w[j] = encode4<FMT>(f[0] * ratio, f[1] * ratio, f[2] * ratio, f[3] * ratio);
                }
                *p = make_uint4(w[0], w[1], w[2], w[3]);
            }
        }
        __syncwarp();                    // every lane has read the scale
    }
    if (lane == 0) *scale = sc;
    const float inv = __fdiv_rn(1.0f, sc);
#pragma unroll
    for (int i = 0; i < N; ++i) {
        const int r = i * RPL + row0;
        if (r < first || r >= last) continue;
        const uint32_t w[4] = {u[i].x, u[i].y, u[i].z, u[i].w};
        float f[8];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            f[2 * j] = __uint_as_float(w[j] << 16) * inv;
            f[2 * j + 1] = __uint_as_float(w[j] & 0xffff0000u) * inv;
        }
        if (FMT == TG_CACHE_INT8 && odd) {
#pragma unroll
            for (int j = 0; j < 8; ++j) f[j] = f[j] != f[j] ? 0.0f : fminf(fmaxf(f[j], -127.0f), 127.0f);
        }
        *reinterpret_cast<uint2*>(codes + r * ld_token + col) =
            make_uint2(encode4<FMT>(f[0], f[1], f[2], f[3]), encode4<FMT>(f[4], f[5], f[6], f[7]));
    }
}

template <int D, int FMT>
__global__ void __launch_bounds__(kWarps * 32) cache_append_q8_kernel(const AppendArgs a) {
    pdl_wait();
    pdl_trigger();
    const int unit = blockIdx.x * kWarps + (threadIdx.x >> 5), lane = threadIdx.x & 31;
    if (unit >= a.units) return;
    const int b = blockIdx.y, Hkv = a.c.Hkv;
    // K's heads, then V's, then the next block
    const int head = unit % Hkv, is_v = unit / Hkv % 2, blk = unit / (2 * Hkv);
    const int64_t len = __ldg(a.c.lengths + b);
    int64_t count = a.n_new;
    bool bad = len < 0 || len > a.c.capacity;
    if (a.counts) {
        const int64_t given = __ldg(a.counts + b);
        count = given < 0 ? 0 : (given > a.n_new ? a.n_new : given);
        bad = bad || count != given;
    }
    const int64_t start = len - count;   // token i goes to slot start + i
    bad = bad || (count > 0 && start < 0);
    if (bad && unit == 0 && lane == 0) atomicOr(a.status, TG_STATUS_CACHE_LENGTH);
    const int64_t lo = start < 0 ? 0 : start, hi = len < a.c.capacity ? len : a.c.capacity;
    const int64_t j = lo / kBlock + blk, s0 = j * kBlock;
    if (lo >= hi || s0 >= hi) return;    // no new token in this block
    const int first = lo > s0 ? static_cast<int>(lo - s0) : 0;
    const int last = hi - s0 < kBlock ? static_cast<int>(hi - s0) : kBlock;
    const int64_t token = s0 + first - start;   // the first of them
    const __nv_bfloat16* x = is_v ? a.v + b * a.ld_v_seq + token * a.ld_v : a.k + b * a.ld_k_seq + token * a.ld_k;
    uint8_t* codes = (is_v ? a.c.v : a.c.k) + b * a.c.ld_seq + s0 * a.c.ld_token + head * D;
    float* scale = (is_v ? a.c.v_scale : a.c.k_scale) + (b * a.c.blocks() + j) * Hkv + head;
    append_block<D, FMT>(x + static_cast<int64_t>(head) * D, is_v ? a.ld_v : a.ld_k, codes, a.c.ld_token, scale, first,
                         last, a.status);
    if (head == 0 && !is_v && lane >= first && lane < last) {
        const int64_t at = b * a.c.capacity + s0 + lane;
        if (a.c.s) a.c.s[at] = a.s_new ? __ldg(a.s_new + b * a.n_new + token + lane - first) : 0.0f;
        if (a.c.w) a.c.w[at] = 0.0f;
    }
}

// ------------------------------------------------------------------------------------------- read
struct ReadArgs {
    Cache c;
    int64_t first, n;
    __nv_bfloat16 *k, *v;
    int tokens;                          // tokens a thread block takes
};

// One thread: 8 codes of K and of V to 16 bytes each, so that a warp's loads and stores are runs of memory; a thread
// block takes `tokens` tokens (about one item a thread: many small thread blocks cover the latency best, 32 tokens a
// thread block took 1.6 times as long for 16 ragged sequences of up to 840).
template <int D, int FMT>
__global__ void __launch_bounds__(kReadThreads) cache_read_q8_kernel(const ReadArgs a) {
    pdl_wait();
    pdl_trigger();
    const int64_t b = blockIdx.y, row0 = static_cast<int64_t>(blockIdx.x) * a.tokens;
    int64_t rows = __ldg(a.c.lengths + b) - a.first;
    if (rows > a.n) rows = a.n;          // (first + n <= capacity)
    rows = rows - row0 < a.tokens ? rows - row0 : a.tokens;
    if (rows <= 0) return;               // (a length far below 0 does not fit an int here)
    const int per_row = a.c.Hkv * (D / 8), items = static_cast<int>(rows) * per_row;
    for (int i = threadIdx.x; i < items; i += kReadThreads) {
        const int r = i / per_row, col = (i - r * per_row) * 8;
        const int64_t slot = a.first + row0 + r;
        const int64_t from = b * a.c.ld_seq + slot * a.c.ld_token + col;
        const int64_t sc = (b * a.c.blocks() + slot / kBlock) * a.c.Hkv + col / D;
        const uint2 ck = __ldg(reinterpret_cast<const uint2*>(a.c.k + from));
        const uint2 cv = __ldg(reinterpret_cast<const uint2*>(a.c.v + from));
        const float sk = __ldg(a.c.k_scale + sc), sv = __ldg(a.c.v_scale + sc);
        const int64_t to = (b * a.n + row0) * a.c.Hkv * D + i * 8ll;
#pragma unroll
        for (int x = 0; x < 2; ++x) {
            const float s = x ? sv : sk;
            float f[4], g[4];
            decode4<FMT>(x ? cv.x : ck.x, f);
            decode4<FMT>(x ? cv.y : ck.y, g);
            *reinterpret_cast<uint4*>((x ? a.v : a.k) + to) =
                make_uint4(pack_bf16x2(f[0] * s, f[1] * s), pack_bf16x2(f[2] * s, f[3] * s),
                           pack_bf16x2(g[0] * s, g[1] * s), pack_bf16x2(g[2] * s, g[3] * s));
        }
    }
}

// ------------------------------------------------------------------------------------------- evict
constexpr int kSelThreads = 1024;
constexpr int kSelWarps = kSelThreads / 32;
constexpr int kCluster = 8;              // thread blocks that select for one long sequence
constexpr int kOneBlockKeys = 24 * 1024; // sequences up to this long: one thread block each
constexpr int kMostKeys = 44 * 1024;     // keys that a thread block's shared memory holds
constexpr int kFew = 256;                // keys that are ranked one by one instead of by two more passes

struct EvictArgs {
    Cache src, dst;
    int64_t budget, sink, recent;
    int32_t* kept;
    unsigned int* status;
    int64_t span;                        // keys that the launch expects of the longest sequence
    int room;                            // keys that its shared memory holds
    int near;                            // whether most of a sequence is expected to stay
};

__device__ __forceinline__ void cluster_st(void* p, uint32_t rank, uint32_t v) {
    asm volatile("st.shared::cluster.u32 [%0], %1;" ::"r"(cluster_addr(p, rank)), "r"(v) : "memory");
}
__device__ __forceinline__ uint32_t cluster_ld(const void* p, uint32_t rank) {
    uint32_t v;
    asm volatile("ld.shared::cluster.u32 %0, [%1];" : "=r"(v) : "r"(cluster_addr(p, rank)) : "memory");
    return v;
}

// Exclusive scan over the block of one value per thread; *total is the block's sum.
template <typename T>
__device__ __forceinline__ T block_scan(T v, T* s_warp, T* total) {
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    T incl = v;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const T y = __shfl_up_sync(0xffffffffu, incl, o);
        if (lane >= o) incl += y;
    }
    if (lane == 31) s_warp[warp] = incl;
    __syncthreads();
    // every warp adds up the warps before it
    T w = s_warp[lane];
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const T y = __shfl_up_sync(0xffffffffu, w, o);
        if (lane >= o) w += y;
    }
    *total = __shfl_sync(0xffffffffu, w, kSelWarps - 1);
    const T before = __shfl_sync(0xffffffffu, w, warp ? warp - 1 : 0);
    return (warp ? before : 0) + incl - v;
}

// CL thread blocks per sequence (one, or a cluster): kept[b, :] ascending, dst's length.  Each thread block owns a
// contiguous part of the tokens between the sinks and the recent ones, its keys in shared memory (where they do not
// fit: read again from L2 each pass), loaded while the sequence's length is still on its way.  A sequence is a few KB
// to a few 100 KB: what bounds the select is the latency of its steps, and in one SM the instructions a key.  So a short
// sequence does without a cluster, whose two barriers a pass with the exchange between them take longer than
// the counting; a thread takes 4 keys at a time; and the loops are short (code that runs once comes from L2
// too: keys in registers, 24 rounds unrolled, took 1.1 us a pass for 9000 keys).
template <int CL>
__global__ void __launch_bounds__(kSelThreads, 1) cache_evict_select_kernel(const EvictArgs a) {
    extern __shared__ __align__(16) uint32_t s_key[];
    __shared__ unsigned s_hist[3][2048];  // one a pass: zero from the start
    __shared__ unsigned s_sum[CL > 1 ? 2048 : 1];   // (the next pass writes it behind a barrier of every reader)
    __shared__ unsigned s_scan[3][kSelWarps];
    __shared__ unsigned long long s_scan2[kSelWarps];
    __shared__ unsigned s_pick[3][3], s_cnt[2];
    __shared__ __align__(16) uint32_t s_few[kFew];
    __shared__ unsigned s_few_n, s_few_pick[2];
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const uint32_t rank = CL > 1 ? cluster_rank_in() : 0;
    for (int i = tid; i < 3 * 2048; i += kSelThreads) s_hist[0][i] = 0u;
    if (tid == 0) s_few_n = 0u;
    pdl_wait();
    pdl_trigger();
    const int b = blockIdx.y, sink = static_cast<int>(a.sink), recent = static_cast<int>(a.recent);
    const int n = length_of(a.src, b, a.status);
    // the keys of this block's part of a span as long as expected (inside the cache, whatever n turns out to be)
    const int expected = static_cast<int>((a.span + CL - 1) / CL);
    const float* w = a.src.w + b * a.src.capacity + sink;
    const int64_t from = static_cast<int64_t>(rank) * expected, end = a.src.capacity - sink - from;
    const int most = end < a.room ? static_cast<int>(end) : a.room;
    float x[8];
    auto load = [&](int i0) {            // 8 keys a thread in one round trip
#pragma unroll
        for (int j = 0; j < 8; ++j)
            if (i0 + kSelThreads * j < most) x[j] = __ldcg(w + from + i0 + kSelThreads * j);
    };
    load(tid);
    int32_t* kept = a.kept + b * a.budget;
    const int gtid = rank * kSelThreads + tid, gthreads = CL * kSelThreads;
    if (gtid == 0) a.dst.lengths[b] = static_cast<int32_t>(n < a.budget ? n : a.budget);
    if (n <= a.budget) {                 // the whole cluster: nothing leaves
        for (int64_t i = gtid; i < a.budget; i += gthreads) kept[i] = i < n ? static_cast<int32_t>(i) : -1;
        return;
    }
    const int budget = static_cast<int>(a.budget), kd = budget - sink - recent;
    // this block's span [c0, c0 + cn) of the m keys, this warp's part [w0, w1) of that in rounds of 128
    const int m = n - sink - recent;
    const bool cached = m <= a.span && expected <= a.room;
    const int per = m <= a.span ? expected : (m + CL - 1) / CL;
    const int c0 = static_cast<int>(min(static_cast<int64_t>(rank) * per, static_cast<int64_t>(m))), cn = min(per, m - c0);
    const int rounds = (per + 4 * kSelThreads - 1) / (4 * kSelThreads);
    const int w0 = min(warp * rounds * 128, cn), w1 = min(w0 + rounds * 128, cn);
    for (int i = gtid; i < sink; i += gthreads) kept[i] = i;
    for (int i = gtid; i < recent; i += gthreads) kept[budget - recent + i] = n - recent + i;
    if (kd == 0) return;
    // keys i .. i + 3 (those before `end`; i a multiple of 4)
    auto four = [&](int i, int end, uint32_t (&k)[4]) {
        if (cached) {
            if (i < end) *reinterpret_cast<uint4*>(k) = *reinterpret_cast<const uint4*>(s_key + i);
        } else {
#pragma unroll
            for (int q = 0; q < 4; ++q)
                if (i + q < end) k[q] = radix_key(__ldcg(w + i + q));
        }
    };
    // a thread's four keys into a histogram: one count where they agree (ties)
    auto count4 = [&](unsigned* hist, const bool (&match)[4], const uint32_t (&digit)[4]) {
        if (match[0] && match[1] && match[2] && match[3] && digit[0] == digit[1] && digit[0] == digit[2] &&
            digit[0] == digit[3]) {
            atomicAdd(&hist[digit[0]], 4u);
        } else {
#pragma unroll
            for (int q = 0; q < 4; ++q)
                if (match[q]) atomicAdd(&hist[digit[q]], 1u);
        }
    };
    __syncthreads();                     // the histograms are zero
    if (cached) {
        // keys to shared memory, and the first pass's count as they come
        for (int i0 = tid; i0 < most; i0 += 8 * kSelThreads) {
            if (i0 != tid) load(i0);
#pragma unroll
            for (int j = 0; j < 8; j += 4) {
                bool match[4];
                uint32_t digit[4];
#pragma unroll
                for (int q = 0; q < 4; ++q) {
                    const int i = i0 + kSelThreads * (j + q);
                    const uint32_t k = i < most ? radix_key(x[j + q]) : 0u;
                    if (i < most) s_key[i] = k;
                    match[q] = i < cn;
                    digit[q] = k >> 21;
                }
                count4(s_hist[0], match, digit);
            }
        }
    }
    w += c0;

    uint32_t prefix = 0, pmask = 0;
    unsigned krem = static_cast<unsigned>(kd);   // rank of the threshold among the keys that match `prefix`
#pragma unroll 1
    for (int p = 0; p < 3; ++p) {
        const int shift = p == 0 ? 21 : (p == 1 ? 10 : 0), nb = p == 2 ? 1024 : 2048;
        for (int i0 = 0; i0 < cn && !(p == 0 && cached); i0 += 4 * kSelThreads) {
            const int i = i0 + 4 * tid;
            uint32_t k[4], digit[4];
            bool match[4];
            four(i, cn, k);
#pragma unroll
            for (int q = 0; q < 4; ++q) {
                match[q] = i + q < cn && (k[q] & pmask) == prefix;
                digit[q] = (k[q] >> shift) & (nb - 1);
            }
            count4(s_hist[p], match, digit);
        }
        const unsigned* hist = s_hist[p];
        if constexpr (CL > 1) {
            // each thread block adds up an eighth of the bins over the cluster and hands it to all
            cluster_sync_all();
            const int sl = nb / CL;
            if (tid < sl) {
                const int bin = rank * sl + tid;
                uint32_t x[CL];
#pragma unroll
                for (int r = 0; r < CL; ++r) x[r] = cluster_ld(&s_hist[p][bin], r);
                uint32_t sum = 0;
#pragma unroll
                for (int r = 0; r < CL; ++r) sum += x[r];
#pragma unroll
                for (int r = 0; r < CL; ++r) cluster_st(&s_sum[bin], r, sum);
            }
            cluster_sync_all();
            hist = s_sum;
        } else {
            __syncthreads();
        }
        // two bins a thread, from the top digit down
        const int d0 = nb - 1 - 2 * tid;
        const unsigned h0 = d0 > 0 ? hist[d0] : 0u, h1 = d0 > 0 ? hist[d0 - 1] : 0u;
        unsigned tot;
        const unsigned e = block_scan(h0 + h1, s_scan[p], &tot);
        if (e < krem && krem <= e + h0) {
            s_pick[p][0] = d0;
            s_pick[p][1] = e;
            s_pick[p][2] = h0;
        } else if (e + h0 < krem && krem <= e + h0 + h1) {
            s_pick[p][0] = d0 - 1;
            s_pick[p][1] = e + h0;
            s_pick[p][2] = h1;
        }
        __syncthreads();
        prefix |= s_pick[p][0] << shift;
        pmask |= static_cast<uint32_t>(nb - 1) << shift;
        krem -= s_pick[p][1];
        if (s_pick[p][2] == krem && prefix) {
            // every key that matches stays: whatever is above prefix - 1
            --prefix;
            krem = 0;
            break;
        }
        if (CL == 1 && p == 0 && s_pick[0][2] <= kFew) {
            // few keys share the threshold's first digit: they are ranked against one another
            for (int i0 = 0; i0 < cn; i0 += 4 * kSelThreads) {
                const int i = i0 + 4 * tid;
                uint32_t k[4];
                four(i, cn, k);
#pragma unroll
                for (int q = 0; q < 4; ++q)
                    if (i + q < cn && (k[q] & pmask) == prefix) s_few[atomicAdd(&s_few_n, 1u)] = k[q];
            }
            __syncthreads();
            const int few = static_cast<int>(s_few_n);
            if (tid < few) {
                const uint32_t k = s_few[tid];
                unsigned above = 0, equal = 0;
#pragma unroll 4
                for (int i = 0; i < few; ++i) {
                    above += s_few[i] > k;
                    equal += s_few[i] == k;
                }
                if (above < krem && krem <= above + equal) {   // (every key equal to it says the same)
                    s_few_pick[0] = k;
                    s_few_pick[1] = krem - above;
                }
            }
            __syncthreads();
            prefix = s_few_pick[0];
            krem = s_few_pick[1];
            break;
        }
    }
    // keys above the threshold `prefix` stay, and the first krem equal to it
    unsigned gt = 0, eq = 0;
    for (int i = w0 + 4 * lane; i < w1; i += 128) {
        uint32_t k[4];
        four(i, w1, k);
#pragma unroll
        for (int q = 0; q < 4; ++q) {
            gt += i + q < w1 && k[q] > prefix;
            eq += i + q < w1 && k[q] == prefix;
        }
    }
    gt = __reduce_add_sync(0xffffffffu, gt);
    eq = __reduce_add_sync(0xffffffffu, eq);
    unsigned long long all;
    unsigned long long mine = block_scan(lane == 0 ? static_cast<unsigned long long>(gt) << 32 | eq : 0ull, s_scan2, &all);
    if constexpr (CL > 1) {
        if (tid == 0) {
            s_cnt[0] = static_cast<unsigned>(all >> 32);
            s_cnt[1] = static_cast<unsigned>(all);
        }
        cluster_sync_all();
        unsigned x = 0, y = 0;           // every warp: the counts of the blocks before this one
        if (lane < static_cast<int>(rank)) {
            x = cluster_ld(&s_cnt[0], lane);
            y = cluster_ld(&s_cnt[1], lane);
        }
        mine += static_cast<unsigned long long>(__reduce_add_sync(0xffffffffu, x)) << 32 |
                __reduce_add_sync(0xffffffffu, y);
    }
    mine = __shfl_sync(0xffffffffu, mine, 0);
    unsigned gt_before = static_cast<unsigned>(mine >> 32), eq_before = static_cast<unsigned>(mine);
    int32_t* to = kept + sink;
    auto one = [&](int i) { return i < w1 ? (cached ? s_key[i] : radix_key(__ldcg(w + i))) : 0u; };
    const unsigned below = (1u << lane) - 1u;
    if (eq == 0 || eq_before >= krem) {  // none of this warp's equal keys stays
        to += min(eq_before, krem);
#pragma unroll 4
        for (int i = w0 + lane; i < w0 + (w1 - w0 + 31) / 32 * 32; i += 32) {
            const bool above = i < w1 && one(i) > prefix;
            const unsigned mg = __ballot_sync(0xffffffffu, above);
            if (above) to[gt_before + __popc(mg & below)] = sink + c0 + i;
            gt_before += __popc(mg);
        }
    } else {
        for (int i = w0 + lane; i < w0 + (w1 - w0 + 31) / 32 * 32; i += 32) {
            const uint32_t k = one(i);
            const bool above = i < w1 && k > prefix, equal = i < w1 && k == prefix;
            const unsigned mg = __ballot_sync(0xffffffffu, above), me = __ballot_sync(0xffffffffu, equal);
            const unsigned g = gt_before + __popc(mg & below), e = eq_before + __popc(me & below);
            if (above || (equal && e < krem)) to[g + min(e, krem)] = sink + c0 + i;
            gt_before += __popc(mg);
            eq_before += __popc(me);
        }
    }
    if (CL > 1) cluster_sync_all();      // no block leaves while a peer may read its shared memory
}

// One warp: one new block of one head, K or V.
template <int D, int FMT>
__global__ void __launch_bounds__(kWarps * 32) cache_evict_gather_kernel(const EvictArgs a) {
    constexpr int LPR = D / 16;          // lanes of a row of codes
    constexpr int RPL = 32 / LPR;
    constexpr int N = kBlock / RPL;
    const int unit = blockIdx.x * kWarps + (threadIdx.x >> 5), lane = threadIdx.x & 31;
    const int Hkv = a.src.Hkv, head = unit % Hkv, is_v = unit / Hkv % 2;
    const int64_t j = unit / (2 * Hkv), b = blockIdx.y;
    if (a.near && j * kBlock < a.budget) {
        // While the select still runs (it began when all that wrote src had ended): this block's share of a sequence
        // of which most will stay, into L2.
        const int64_t n = min(max(static_cast<int64_t>(__ldg(a.src.lengths + b)), static_cast<int64_t>(0)), a.src.capacity);
        const int64_t r0 = j * kBlock * n / a.budget, r1 = min((j + 1) * kBlock * n / a.budget, n);
        const uint8_t* p = (is_v ? a.src.v : a.src.k) + b * a.src.ld_seq + head * D;
        for (int64_t r = r0 + lane; r < r1; r += 32)
            asm volatile("prefetch.global.L2 [%0];" ::"l"(p + r * a.src.ld_token));
    }
    pdl_wait();
    pdl_trigger();
    if (j * kBlock >= a.budget) return;
    const int slot = j * kBlock + lane < a.budget ? a.kept[b * a.budget + j * kBlock + lane] : -1;
    if (!__any_sync(0xffffffffu, slot >= 0)) return;
    const uint8_t* from = (is_v ? a.src.v : a.src.k) + b * a.src.ld_seq + head * D + (lane % LPR) * 16;
    const float* from_scale = (is_v ? a.src.v_scale : a.src.k_scale) + b * a.src.blocks() * Hkv + head;
    const float mine = slot >= 0 ? __ldg(from_scale + static_cast<int64_t>(slot / kBlock) * Hkv) : 0.0f;
    uint4 u[N];
#pragma unroll
    for (int i = 0; i < N; ++i) {
        const int r = i * RPL + lane / LPR;
        const int at = __shfl_sync(0xffffffffu, slot, r);
        u[i] = at >= 0 ? __ldg(reinterpret_cast<const uint4*>(from + at * a.src.ld_token)) : make_uint4(0u, 0u, 0u, 0u);
    }
    float amax = 0.0f;
#pragma unroll
    for (int i = 0; i < N; ++i) {
        // the largest magnitude of a row's codes: their own order (NaN codes do not count)
        const uint32_t w[4] = {u[i].x, u[i].y, u[i].z, u[i].w};
        uint32_t top = 0;
#pragma unroll
        for (int x = 0; x < 4; ++x) {
            uint32_t c;
            if constexpr (FMT == TG_CACHE_E4M3) {
                c = w[x] & 0x7f7f7f7fu;
                c &= ~__vcmpeq4(c, 0x7f7f7f7fu);
            } else {
                c = __vabs4(w[x]);
            }
            top = __vmaxu4(top, c);
        }
        top = __vmaxu4(top, top >> 16);
        top = __vmaxu4(top, top >> 8) & 0xffu;
        float f[4];
        if constexpr (FMT == TG_CACHE_E4M3)
            decode4<FMT>(top, f);
        else
            f[0] = static_cast<float>(top);
        amax = fmaxf(amax, f[0] * __shfl_sync(0xffffffffu, mine, i * RPL + lane / LPR));
    }
    const float scale = scale_for<FMT>(warp_max(amax));
    uint8_t* to = (is_v ? a.dst.v : a.dst.k) + b * a.dst.ld_seq + j * kBlock * a.dst.ld_token + head * D +
                  (lane % LPR) * 16;
#pragma unroll
    for (int i = 0; i < N; ++i) {
        const int r = i * RPL + lane / LPR;
        const int at = __shfl_sync(0xffffffffu, slot, r);
        uint32_t w[4] = {u[i].x, u[i].y, u[i].z, u[i].w};
        const float before = __shfl_sync(0xffffffffu, mine, r);
        if (before != scale) {
            // A row with a code other than 0 has before <= qmax / (the least code) scale: below kMostRatio.  One of
            // zeros may come from any scale, and 0 times an infinite ratio is not 0.
            const float ratio = fminf(__fdiv_rn(before, scale), kMostRatio);
#pragma unroll
            for (int x = 0; x < 4; ++x) {
                float f[4];
                decode4<FMT>(w[x], f);
                w[x] = encode4<FMT>(f[0] * ratio, f[1] * ratio, f[2] * ratio, f[3] * ratio);
            }
        }
        if (at >= 0) *reinterpret_cast<uint4*>(to + r * a.dst.ld_token) = make_uint4(w[0], w[1], w[2], w[3]);
    }
    if (lane == 0) (is_v ? a.dst.v_scale : a.dst.k_scale)[(b * a.dst.blocks() + j) * Hkv + head] = scale;
    if (head == 0 && !is_v && slot >= 0) {
        const int64_t at = b * a.dst.capacity + j * kBlock + lane, of = b * a.src.capacity + slot;
        if (a.dst.s) a.dst.s[at] = a.src.s ? a.src.s[of] : 0.0f;
        if (a.dst.w) a.dst.w[at] = a.src.w[of];
    }
}

template <int CL>
static tg_status launch_select(EvictArgs a, int64_t keys, cudaStream_t st) {
    static std::atomic<int> smem_set[64];
    auto kern = cache_evict_select_kernel<CL>;
    constexpr int kMost = CL == 1 ? kOneBlockKeys : kMostKeys;   // multiples of 4
    if (!set_max_dynamic_smem(kern, kMost * 4, smem_set)) return TG_ERR_CUDA;
    a.span = keys > 0 ? keys : 0;
    const int64_t per = (a.span + CL - 1) / CL;
    a.room = per <= kMost ? static_cast<int>((per + 3) / 4 * 4) : 0;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(CL, static_cast<unsigned>(a.src.batch));
    cfg.blockDim = dim3(kSelThreads);
    cfg.dynamicSmemBytes = static_cast<size_t>(a.room) * 4;
    cfg.stream = st;
    cudaLaunchAttribute at[2] = {pdl_attr()};
    at[1].id = cudaLaunchAttributeClusterDimension;
    at[1].val.clusterDim.x = CL;
    at[1].val.clusterDim.y = 1;
    at[1].val.clusterDim.z = 1;
    cfg.attrs = at;
    cfg.numAttrs = CL > 1 ? 2 : 1;
    return cudaLaunchKernelEx(&cfg, kern, a) == cudaSuccess ? launch_status() : TG_ERR_CUDA;
}

static size_t code_bytes(const Cache& c, int d) {
    if (c.batch == 0 || c.capacity == 0) return 0;
    return static_cast<size_t>(c.batch - 1) * c.ld_seq + static_cast<size_t>(c.capacity - 1) * c.ld_token +
           static_cast<size_t>(c.Hkv) * d;
}

}  // namespace q8
}  // namespace tg

using namespace tg;

extern "C" tg_status tg_cache_append_q8(const tg_cache_q8* cache, const tg_bf16* k, int64_t ld_k, int64_t ld_k_seq,
                                        const tg_bf16* v, int64_t ld_v, int64_t ld_v_seq, int64_t n_new,
                                        const int32_t* counts, const float* s_new, void* workspace,
                                        size_t workspace_bytes, void* stream) {
    q8::AppendArgs a = {};
    const tg_status ok = q8::check_cache(cache, &a.c);
    if (ok != TG_OK) return ok;
    if (n_new < 0) return TG_ERR_INVALID_ARG;
    if (n_new > 0x7fffffffLL) return TG_ERR_UNSUPPORTED;
    if (n_new == 0 || a.c.batch == 0 || a.c.capacity == 0) return TG_OK;
    if (!k || !v || !workspace || !aligned16(k) || !aligned16(v) || !aligned16(workspace)) return TG_ERR_INVALID_ARG;
    if (workspace_bytes < kWsHeader) return TG_ERR_INVALID_ARG;
    const int64_t row = static_cast<int64_t>(a.c.Hkv) * cache->d_h;
    if (((ld_k | ld_v | ld_k_seq | ld_v_seq) % 8) != 0) return TG_ERR_INVALID_ARG;
    if (n_new > 1 && (ld_k < row || ld_v < row)) return TG_ERR_INVALID_ARG;
    if (a.c.batch > 1 && (ld_k_seq < row || ld_v_seq < row)) return TG_ERR_INVALID_ARG;
    a.k = reinterpret_cast<const __nv_bfloat16*>(k);
    a.v = reinterpret_cast<const __nv_bfloat16*>(v);
    a.ld_k = ld_k;
    a.ld_v = ld_v;
    a.ld_k_seq = ld_k_seq;
    a.ld_v_seq = ld_v_seq;
    a.n_new = n_new;
    a.counts = counts;
    a.s_new = s_new;
    a.status = status_word(workspace);
    // blocks that n tokens in a row touch at most, wherever they begin
    int64_t blocks = (n_new + q8::kBlock - 2) / q8::kBlock + 1;
    const int64_t all = a.c.capacity / q8::kBlock;
    if (blocks > all) blocks = all;
    const int64_t units = blocks * a.c.Hkv * 2;
    if (units > 0x7fffff00LL) return TG_ERR_UNSUPPORTED;
    a.units = static_cast<int>(units);
    const dim3 grid(static_cast<unsigned>((units + q8::kWarps - 1) / q8::kWarps), static_cast<unsigned>(a.c.batch));
    auto kern = cache->d_h == 128
                    ? (cache->format == TG_CACHE_E4M3 ? q8::cache_append_q8_kernel<128, TG_CACHE_E4M3>
                                                      : q8::cache_append_q8_kernel<128, TG_CACHE_INT8>)
                    : (cache->format == TG_CACHE_E4M3 ? q8::cache_append_q8_kernel<64, TG_CACHE_E4M3>
                                                      : q8::cache_append_q8_kernel<64, TG_CACHE_INT8>);
    return q8::launch_pdl(kern, grid, dim3(q8::kWarps * 32), 0, as_stream(stream), a);
}

extern "C" tg_status tg_cache_read_q8(const tg_cache_q8* cache, int64_t first, int64_t n, tg_bf16* k_out,
                                      tg_bf16* v_out, void* stream) {
    q8::ReadArgs a = {};
    const tg_status ok = q8::check_cache(cache, &a.c);
    if (ok != TG_OK) return ok;
    if (first < 0 || n < 0 || first > a.c.capacity || n > a.c.capacity - first) return TG_ERR_INVALID_ARG;
    if (n == 0 || a.c.batch == 0) return TG_OK;
    if (!k_out || !v_out || !aligned16(k_out) || !aligned16(v_out)) return TG_ERR_INVALID_ARG;
    a.first = first;
    a.n = n;
    a.k = reinterpret_cast<__nv_bfloat16*>(k_out);
    a.v = reinterpret_cast<__nv_bfloat16*>(v_out);
    const int per_row = a.c.Hkv * (cache->d_h / 8);
    a.tokens = per_row < q8::kReadThreads ? q8::kReadThreads / per_row : 1;
    const dim3 grid(static_cast<unsigned>((n + a.tokens - 1) / a.tokens), static_cast<unsigned>(a.c.batch));
    auto kern = cache->d_h == 128 ? (cache->format == TG_CACHE_E4M3 ? q8::cache_read_q8_kernel<128, TG_CACHE_E4M3>
                                                                    : q8::cache_read_q8_kernel<128, TG_CACHE_INT8>)
                                  : (cache->format == TG_CACHE_E4M3 ? q8::cache_read_q8_kernel<64, TG_CACHE_E4M3>
                                                                    : q8::cache_read_q8_kernel<64, TG_CACHE_INT8>);
    return q8::launch_pdl(kern, grid, dim3(q8::kReadThreads), 0, as_stream(stream), a);
}

extern "C" tg_status tg_cache_evict_q8(const tg_cache_q8* src, const tg_cache_q8* dst, int64_t budget, int64_t sink,
                                       int64_t recent, int64_t max_len, int32_t* kept, void* workspace,
                                       size_t workspace_bytes, void* stream) {
    q8::EvictArgs a = {};
    tg_status ok = q8::check_cache(src, &a.src);
    if (ok == TG_OK) ok = q8::check_cache(dst, &a.dst);
    if (ok != TG_OK) return ok;
    if (src->format != dst->format || src->batch != dst->batch || src->Hkv != dst->Hkv || src->d_h != dst->d_h)
        return TG_ERR_INVALID_ARG;
    if (budget < 0 || sink < 0 || recent < 0 || max_len < 0 || sink > budget || recent > budget - sink ||
        budget > dst->capacity)
        return TG_ERR_INVALID_ARG;
    if (src->batch == 0) return TG_OK;
    if (!workspace || !aligned16(workspace) || workspace_bytes < kWsHeader || (budget > 0 && !kept) ||
        (src->capacity > 0 && !src->w))
        return TG_ERR_INVALID_ARG;
    const size_t sb = q8::code_bytes(a.src, src->d_h), db = q8::code_bytes(a.dst, dst->d_h);
    const size_t st_bytes = static_cast<size_t>(src->batch) * src->capacity * 4, sc_bytes = st_bytes / q8::kBlock * src->Hkv;
    const size_t dt_bytes = static_cast<size_t>(dst->batch) * dst->capacity * 4, dc_bytes = dt_bytes / q8::kBlock * dst->Hkv;
    const size_t len_bytes = static_cast<size_t>(src->batch) * 4;
    if (q8::overlap(src->k, sb, dst->k, db) || q8::overlap(src->v, sb, dst->v, db) ||
        q8::overlap(src->k, sb, dst->v, db) || q8::overlap(src->v, sb, dst->k, db) ||
        q8::overlap(src->w, st_bytes, dst->w, dt_bytes) || q8::overlap(src->s, st_bytes, dst->s, dt_bytes) ||
        q8::overlap(src->k_scale, sc_bytes, dst->k_scale, dc_bytes) ||
        q8::overlap(src->v_scale, sc_bytes, dst->v_scale, dc_bytes) ||
        q8::overlap(src->lengths, len_bytes, dst->lengths, len_bytes))
        return TG_ERR_INVALID_ARG;
    a.budget = budget;
    a.sink = sink;
    a.recent = recent;
    a.kept = kept;
    a.status = status_word(workspace);
    if (max_len == 0 || max_len > src->capacity) max_len = src->capacity;
    cudaStream_t st = as_stream(stream);
    tg_status r;
    a.near = max_len <= 2 * budget;
    const int64_t keys = max_len - sink - recent;
    r = keys <= q8::kOneBlockKeys ? q8::launch_select<1>(a, keys, st) : q8::launch_select<q8::kCluster>(a, keys, st);
    if (r != TG_OK || budget == 0) return r;
    const int64_t units = (budget + q8::kBlock - 1) / q8::kBlock * src->Hkv * 2;
    const dim3 grid(static_cast<unsigned>((units + q8::kWarps - 1) / q8::kWarps), static_cast<unsigned>(src->batch));
    auto kern = src->d_h == 128 ? (src->format == TG_CACHE_E4M3 ? q8::cache_evict_gather_kernel<128, TG_CACHE_E4M3>
                                                                : q8::cache_evict_gather_kernel<128, TG_CACHE_INT8>)
                                : (src->format == TG_CACHE_E4M3 ? q8::cache_evict_gather_kernel<64, TG_CACHE_E4M3>
                                                                : q8::cache_evict_gather_kernel<64, TG_CACHE_INT8>);
    return q8::launch_pdl(kern, grid, dim3(q8::kWarps * 32), 0, st, a);
}
