// route.cu — expert routing: the k largest logits of each token, their weights, every
// expert's rows, the balance loss, and the gradient of weights and loss by the logits.
//
// The expert layers' products (fp8_block_gemm_grouped and its weight gradient) read rows
// sorted by expert and each group's first row; these kernels make both from the logits.
//
//   p = softmax(l), chosen = the k largest l;  weight_j = p_j (or p_j / sum of the chosen p)
//   loss = sum_e slope_e sum_t p_te,  slope_e = E counts_e / (C N)
//   dl = p (dp - <p, dp>),  dp_e = dloss slope_e + (chosen: dw_j, or (dw_j - <dw, w>) / sum of the chosen p)
//
// Rows are given out without atomics whose order matters: a group of lanes walks a run of
// tokens in order and counts per expert in shared memory; prefixes over the runs of a CTA,
// then over the CTAs, turn the counts into rows.  Sums of probabilities add up in the same
// fixed order.
#include "block.cuh"

namespace fp8dl {

namespace rt {
constexpr int MAX_TILES = 160;  // CTAs of the first kernel (workspace rows); one per SM fits every GB300
constexpr int MAX_K = 32;       // choices of a token: one per lane
constexpr int KEPT = 8;         // a run's first tokens, whose choices wait in shared memory for their rows
constexpr float NEG_INF = -__builtin_huge_valf();
}

struct RouteArgs {
    const void *logits;
    int64_t tokens;
    int experts, k, normalize, vec;
    const uint8_t *valid;
    int32_t *expert, *position, *token, *offsets, *counts;
    float *weight, *slope, *loss;
    int32_t *hist;     // [tiles][experts]: the tile's choices of each expert
    int32_t *counted;  // [tiles]: its tokens with a choice
    float *psum;       // [tiles][experts]: its sums of p, or NULL
    int64_t per;    // tokens of a run
};

// Order-preserving key of a float, 0 for what is never chosen (-infinity, NaN); -0 counts as 0.
__device__ __forceinline__ uint32_t route_key(float v) {
    const uint32_t b = __float_as_uint(v + 0.0f);
    return v > rt::NEG_INF ? b ^ ((uint32_t)((int32_t)b >> 31) | 0x80000000u) : 0u;
}
__device__ __forceinline__ float route_value(uint32_t key) {
    return __uint_as_float(key & 0x80000000u ? key ^ 0x80000000u : ~key);
}
// The same of two bf16 values at once: a 16-bit key in the upper half of each, and the expert's place from the end below
// it: no two are alike, and the largest is the largest logit of the lowest expert.  -infinity's key (NaN's too) is below
// NONE16, every other one above it.
constexpr uint32_t NONE16 = 0x00800000u;
__device__ __forceinline__ void route_keys16(uint32_t pair, int i, uint32_t &lo, uint32_t &hi) {
    uint32_t y, sign;
    asm("{.reg .b32 a;\n\tadd.rn.bf16x2 a, %1, %2;\n\tmax.bf16x2 %0, a, %3;}" : "=r"(y) : "r"(pair), "r"(0u), "r"(0xff80ff80u));
    asm("prmt.b32 %0, %1, 0, 0xbb99;" : "=r"(sign) : "r"(y));  // all ones in the halves below zero
    y ^= sign | 0x80008000u;
    lo = __byte_perm(y, 0xffffu - i, 0x1054), hi = (y & 0xffff0000u) | (0xfffeu - i);
}
__device__ __forceinline__ float route_value16(uint32_t key) {
    return __uint_as_float(key & 0x80000000u ? (key & 0xffff0000u) ^ 0x80000000u : ~key & 0xffff0000u);
}
// exp(v - m) from the hardware's 2^x: v - m first, so that the error goes by that difference (2 units of 2^-24 for each
// 1 of it, and 4 of 2^x) whatever the logits' size.
__device__ __forceinline__ float route_exp(float v, float m) { return ex2_approx_ftz((v - m) * 1.4426950409f); }

// S (1, 2, 4 or 8) keys into descending order: Batcher's odd-even merge exchange (19 exchanges for eight).
template <typename T>
__device__ __forceinline__ void exchange_down(T &a, T &b) {
    const T hi = a > b ? a : b, lo = a > b ? b : a;
    a = hi, b = lo;
}
template <typename T, int S>
__device__ __forceinline__ void sort_down(T (&k)[S]) {
#pragma unroll
    for (int p = 1; p < S; p *= 2)
#pragma unroll
        for (int q = p; q >= 1; q /= 2)
#pragma unroll
            for (int j = q % p; j + q < S; j += 2 * q)
#pragma unroll
                for (int i = 0; i < q; i++)
                    if (i + j + q < S && (i + j) / (2 * p) == (i + j + q) / (2 * p)) exchange_down(k[i + j], k[i + j + q]);
}

// S consecutive logits of a row from element i0 on, as they lie in memory (lane-contiguous, so that the lowest lane
// among equal maxima holds the lowest expert); -infinity behind the row's end.
template <int XKIND, int S>
struct Logits {
    static constexpr int ESZ = XKIND == FP8DL_BF16 ? 2 : 4, BYTES = S * ESZ, WORDS = (BYTES + 3) / 4, PAIRS = (S + 1) / 2;
    uint32_t w[WORDS];
    __device__ __forceinline__ void none() {
#pragma unroll
        for (int q = 0; q < WORDS; q++) w[q] = XKIND == FP8DL_BF16 ? 0xff80ff80u : 0xff800000u;
    }
    __device__ __forceinline__ void load(const char *p, int E, int i0, bool vec) {  // p: logit i0 of a row of E
        none();
        if (vec && BYTES >= 4) {
            if (i0 >= E) return;  // E is a multiple of S: all of the lane's or none
            if constexpr (BYTES >= 16) {
#pragma unroll
                for (int q = 0; q < BYTES / 16; q++) {
                    const uint4 u = *reinterpret_cast<const uint4 *>(p + 16 * q);
                    w[4 * q] = u.x, w[4 * q + 1] = u.y, w[4 * q + 2] = u.z, w[4 * q + 3] = u.w;
                }
            } else if constexpr (BYTES == 8) {
                const uint2 u = *reinterpret_cast<const uint2 *>(p);
                w[0] = u.x, w[1] = u.y;
            } else if constexpr (BYTES == 4) {
                w[0] = *reinterpret_cast<const uint32_t *>(p);
            }
        } else {
#pragma unroll
            for (int s = 0; s < S; s++) {
                if (i0 + s >= E) continue;
                if (XKIND == FP8DL_F32) w[s < WORDS ? s : 0] = reinterpret_cast<const uint32_t *>(p)[s];
                else w[s / 2] = __byte_perm(w[s / 2], reinterpret_cast<const uint16_t *>(p)[s], s & 1 ? 0x5410 : 0x3254);
            }
        }
    }
    __device__ __forceinline__ float2 pair(int p) const {
        if (XKIND == FP8DL_BF16) return make_float2(bf16_lo(w[p]), bf16_hi(w[p]));
        return make_float2(__uint_as_float(w[2 * p < WORDS ? 2 * p : 0]), S > 1 ? __uint_as_float(w[2 * p + 1 < WORDS ? 2 * p + 1 : 0]) : rt::NEG_INF);
    }
};

// exp(v - m) of a pair, by the same steps as route_exp.
__device__ __forceinline__ float2 route_exp2(float2 v, float m) {
    const float2 x = __fmul2_rn(__fadd2_rn(v, f2(-m)), f2(1.4426950409f));
    return make_float2(ex2_approx_ftz(x.x), ex2_approx_ftz(x.y));
}

// The largest of a group's values, the same in all of its lanes; NaN does not count.
__device__ __forceinline__ float group_max(float v, uint32_t mask) {
    float m;
    asm volatile("redux.sync.max.f32 %0, %1, %2;" : "=f"(m) : "f"(v), "r"(mask));
    return m;
}

// Sum over the G lanes of a group, the same in all of them.
template <int G>
__device__ __forceinline__ float group_sum(float v) {
#pragma unroll
    for (int o = G / 2; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
    return v;
}

// Exclusive prefix sums of total[0 .. n) into first[0 .. n], by all threads of a block of THREADS
// >= 32 threads (a multiple of 32); n <= 1024.  `warps` holds THREADS / 32 entries.
template <int THREADS>
__device__ __forceinline__ void scan_experts(const int32_t *total, int32_t *first, int n, int32_t *warps) {
    constexpr int PER = 1024 / THREADS;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, i0 = threadIdx.x * PER;
    int32_t own[PER], sum = 0;
#pragma unroll
    for (int i = 0; i < PER; i++) {
        own[i] = i0 + i < n ? total[i0 + i] : 0;
        sum += own[i];
    }
    int32_t run = sum;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int32_t u = __shfl_up_sync(0xffffffffu, run, o);
        if (lane >= o) run += u;
    }
    if (lane == 31) warps[warp] = run;
    __syncthreads();
    int32_t before = run - sum + __reduce_add_sync(0xffffffffu, lane < warp ? warps[lane] : 0);
#pragma unroll
    for (int i = 0; i < PER; i++) {
        if (i0 + i < n) first[i0 + i] = before;
        before += own[i];
        if (i0 + i == n - 1) first[n] = before;
    }
    __syncthreads();
}

// slope and loss from every expert's count and sum of p, by a block of THREADS threads.
template <int THREADS>
__device__ __forceinline__ void balance(const RouteArgs &a, const int32_t *total, const float *p, int counted, int choices,
                                        float *warps) {
    const float unit = counted > 0 ? __fdiv_rn((float)a.experts, (float)choices * (float)counted) : 0.0f;
    float sum = 0.0f;
    for (int e = threadIdx.x; e < a.experts; e += THREADS) {
        const float s = (float)total[e] * unit;
        a.slope[e] = s;
        sum = fmaf(s, p[e], sum);
    }
    sum = group_sum<32>(sum);
    if ((threadIdx.x & 31) == 0) warps[threadIdx.x >> 5] = sum;
    __syncthreads();
    if (threadIdx.x < 32) {
        sum = group_sum<32>(threadIdx.x < THREADS / 32 ? warps[threadIdx.x] : 0.0f);
        if (threadIdx.x == 0) a.loss[0] = sum;
    }
}

// One CTA routes a tile of tokens: G lanes a token, lane l the experts l S .. l S + S - 1, a run of
// a.per consecutive tokens per group of lanes; the next token's logits are under way meanwhile.
//   choice   each lane sorts its keys once (up to eight; more: it searches them again); k rounds of a maximum over
//            the lanes (redux) of the lanes' first keys, and the lane that had it moves up.  Lane j keeps choice j.
//   row      rank within the run from the CTA's shared counters (a token's experts differ, so its
//            lanes never meet), plus the runs before it after the last token.  The ranks of a run's first
//            tokens wait in shared memory, further ones in `position`.
//   SINGLE   the tile is all there is: rows, counts and the loss are finished here, one launch.
// The runs' counters and then the runs' sums of p share one buffer [runs][experts].
// Bound: the issue slots (about 390 instructions a token of 256 experts and 8 choices, 66% of the slots in use, half of
// them the one pipe of comparisons and selects); few tokens: the launches.  32768 tokens of 256 experts in bf16, 8 choices,
// this kernel and the next: 23 us with the balance loss, 21 without (fp32 33); 1 token of 64: 3.2 us.
template <int XKIND, int G, int S, int THREADS, bool SINGLE>
__global__ void __launch_bounds__(THREADS) route_kernel(const RouteArgs a) {
    constexpr int NG = THREADS / G;
    extern __shared__ int32_t cnt[];
    __shared__ int32_t total[SINGLE ? 1024 : 1], first[SINGLE ? 1025 : 1], warps[THREADS / 32], counted;
    const int E = a.experts, k = a.k, tid = threadIdx.x, lane = tid & 31, run = tid / G, l = tid % G;
    const uint32_t gmask = G == 32 ? 0xffffffffu : ((1u << (G & 31)) - 1u) << (lane & ~(G - 1));
    pdl_wait();
    pdl_trigger();
    const int64_t tile0 = (int64_t)blockIdx.x * NG * a.per, t0 = tile0 + run * a.per;
    const int runs = (int)min((a.tokens - tile0 + a.per - 1) / a.per, (int64_t)NG);  // those that have tokens
    for (int i = tid; i < runs * E; i += THREADS) cnt[i] = 0;
    if (tid == 0) counted = 0;
    __syncthreads();
    int32_t *mine = cnt + run * E;
    constexpr int PAIRS = Logits<XKIND, S>::PAIRS;
    float2 ps[PAIRS];
#pragma unroll
    for (int p = 0; p < PAIRS; p++) ps[p] = f2(0.0f);
    int n_counted = 0;
    Logits<XKIND, S> x, x_next;
    // tokens * k is below 2^31: so are the tokens of a run, and the places of their choices
    const int per = (int)a.per, n_here = (int)min(max(a.tokens - t0, (int64_t)0), a.per);
    const int row = E * Logits<XKIND, S>::ESZ;
    const char *at_logits = static_cast<const char *>(a.logits) + t0 * row + l * S * Logits<XKIND, S>::ESZ;
    const uint8_t *at_valid = a.valid ? a.valid + t0 : nullptr;
    const auto load = [&](int i) {  // of token i of the run, one after the other: -infinity where there is none
        if (i < n_here && (!at_valid || at_valid[i])) x_next.load(at_logits, E, l * S, a.vec);
        else x_next.none();
        at_logits += row;
    };
    load(0);
    const int kept_tokens = min(per, rt::KEPT);
    int32_t *kept = cnt + NG * E;  // [token of the run][run][choice]: the expert and the rank in the run above it, or -1
    uint32_t place = (uint32_t)(t0 * k) + l;
    for (int i = 0; i < per; i++, place += k) {
        const bool here = i < n_here;
        uint32_t key[S], best = 0, choice = 0;  // choice: lane j's, the key of choice j
        int32_t pick = -1;                      // and its expert
        int slot = 0;
        x = x_next;
#pragma unroll
        for (int p = 0; p < PAIRS; p++) {
            uint32_t lo, hi;
            if (XKIND == FP8DL_BF16) route_keys16(x.w[p < Logits<XKIND, S>::WORDS ? p : 0], l * S + 2 * p, lo, hi);
            else lo = route_key(x.pair(p).x), hi = route_key(x.pair(p).y);
            key[2 * p] = lo;
            if (2 * p + 1 < S) key[2 * p + 1 < S ? 2 * p + 1 : 0] = hi;
        }
        if (S < 16) load(i + 1);  // under way while this token's experts are chosen
        if (XKIND == FP8DL_BF16 && S <= 8) {  // the lane's keys in order once; the lane that had the largest moves up
            sort_down(key);
            if (k <= S) {  // S - j keys of a lane still matter at choice j
#pragma unroll
                for (int j = 0; j < S; j++) {
                    if (j >= k) break;
                    const uint32_t top = __reduce_max_sync(gmask, key[0]);
                    if (l == j) choice = top;
                    const bool taken = key[0] == top;
#pragma unroll
                    for (int s = 0; s + 1 < S - j; s++) key[s] = taken ? key[s + 1] : key[s];
                }
            } else {
                for (int j = 0; j < k; j++) {
                    const uint32_t top = __reduce_max_sync(gmask, key[0]);
                    if (l == j) choice = top;
                    const bool taken = key[0] == top;
#pragma unroll
                    for (int s = 0; s < S; s++) key[s] = taken ? (s + 1 < S ? key[s + 1 < S ? s + 1 : s] : 0u) : key[s];
                }
            }
        } else if (XKIND == FP8DL_BF16) {
#pragma unroll
            for (int s = 0; s < S; s++) best = max(best, key[s]);
            for (int j = 0; j < k; j++) {
                const uint32_t top = __reduce_max_sync(gmask, best);
                if (l == j) choice = top;
                if (best == top) {  // one lane: the largest of its keys below it
                    best = 0;
#pragma unroll
                    for (int s = 0; s < S; s++) best = max(best, key[s] < top ? key[s] : 0u);
                }
            }
        } else if (S <= 8) {  // the same with the expert's place beside an fp32's key; of lanes with the largest the lowest moves up
            uint64_t list[S];
#pragma unroll
            for (int s = 0; s < S; s++) list[s] = (uint64_t)key[s] << 32 | (uint32_t)(0xffff - (l * S + s));
            sort_down(list);
            const auto take = [&](int j) {
                const uint32_t own = (uint32_t)(list[0] >> 32), top = __reduce_max_sync(gmask, own);
                const int winner = __ffs(__ballot_sync(0xffffffffu, own == top) & gmask) - 1;
                const uint32_t place_of = __shfl_sync(0xffffffffu, (uint32_t)list[0], winner);
                if (l == j && top != 0) {
                    choice = top;
                    pick = 0xffff - (int)place_of;
                }
                return lane == winner;
            };
            if (k <= S) {
#pragma unroll
                for (int j = 0; j < S; j++) {
                    if (j >= k) break;
                    const bool taken = take(j);
#pragma unroll
                    for (int s = 0; s + 1 < S - j; s++) list[s] = taken ? list[s + 1] : list[s];
                }
            } else {
                for (int j = 0; j < k; j++) {
                    const bool taken = take(j);
#pragma unroll
                    for (int s = 0; s < S; s++) list[s] = taken ? (s + 1 < S ? list[s + 1 < S ? s + 1 : s] : 0u) : list[s];
                }
            }
        } else {
#pragma unroll
            for (int s = S - 1; s >= 0; s--)
                if (key[s] >= best) best = key[s], slot = s;
            for (int j = 0; j < k; j++) {
                const uint32_t top = __reduce_max_sync(gmask, best);
                const int winner = __ffs(__ballot_sync(0xffffffffu, best == top) & gmask) - 1;
                const int where = __shfl_sync(0xffffffffu, slot, winner);
                if (l == j && top != 0) {
                    choice = top;
                    pick = (winner & (G - 1)) * S + where;
                }
                if (lane == winner) {
                    best = 0;
#pragma unroll
                    for (int s = S - 1; s >= 0; s--) {
                        if (s == where) key[s] = 0;
                        if (key[s] >= best) best = key[s], slot = s;
                    }
                }
            }
        }
        if (XKIND == FP8DL_BF16) {
            if (choice < NONE16) choice = 0;
            else pick = 0xffff - (int)(choice & 0xffff);
        }
        const uint32_t top = __shfl_sync(0xffffffffu, choice, lane & ~(G - 1));
        const auto value = [](uint32_t c) { return XKIND == FP8DL_BF16 ? route_value16(c) : route_value(c); };
        const float m = top ? value(top) : 0.0f;  // nothing to choose: all -infinity or NaN, whose exponentials are 0 or NaN
        float2 v[PAIRS], z2 = f2(0.0f);
#pragma unroll
        for (int p = 0; p < PAIRS; p++) {
            v[p] = route_exp2(x.pair(p), m);
            z2 = __fadd2_rn(z2, v[p]);
        }
        const float z = group_sum<G>(z2.x + z2.y), inv = top ? __frcp_rn(z) : 1.0f;
#pragma unroll
        for (int p = 0; p < PAIRS; p++) ps[p] = __ffma2_rn(v[p], f2(inv), ps[p]);
        const float e = pick >= 0 ? route_exp(value(choice), m) : 0.0f;
        const float chosen = group_sum<G>(e);
        if (l == 0 && top) n_counted++;
        if (S >= 16) load(i + 1);
        if (here && l < k) {
            float w = 0.0f;
            int32_t rank = -1;
            if (pick >= 0) {
                w = z == z ? e * (a.normalize ? __frcp_rn(chosen) : inv) : z;
                rank = mine[pick];
                mine[pick] = rank + 1;
            }
            a.expert[place] = pick;
            a.weight[place] = w;
            if (i < kept_tokens) kept[(i * NG + run) * k + l] = pick >= 0 ? rank << 10 | pick : -1;
            else a.position[place] = rank;
        }
        __syncwarp();
    }
    if (n_counted) atomicAdd(&counted, n_counted);
    __syncthreads();
    int32_t *sums = SINGLE ? total : a.hist + (int)blockIdx.x * E;
    if (G == 32) {  // the runs before each run: 16 or 32 of them, a thread per expert
        for (int e = tid; e < E; e += THREADS) {
            int32_t sum = 0;
            for (int g0 = 0; g0 < runs; g0 += 8) {  // eight reads at once
                int32_t c[8];
#pragma unroll
                for (int i = 0; i < 8; i++) c[i] = g0 + i < runs ? cnt[(g0 + i) * E + e] : 0;
#pragma unroll
                for (int i = 0; i < 8; i++) {
                    if (g0 + i < runs) cnt[(g0 + i) * E + e] = sum;
                    sum += c[i];
                }
            }
            sums[e] = sum;
        }
    } else {  // 64 or 128 runs, a warp per expert
        for (int e = tid >> 5; e < E; e += THREADS / 32) {
            int32_t sum = 0;
            for (int g0 = 0; g0 < runs; g0 += 32) {
                const bool ok = g0 + lane < runs;
                const int32_t c = ok ? cnt[(g0 + lane) * E + e] : 0;
                int32_t upto = c;
#pragma unroll
                for (int o = 1; o < 32; o <<= 1) {
                    const int32_t u = __shfl_up_sync(0xffffffffu, upto, o);
                    if (lane >= o) upto += u;
                }
                if (ok) cnt[(g0 + lane) * E + e] = sum + upto - c;
                sum += __shfl_sync(0xffffffffu, upto, 31);
            }
            if (lane == 0) sums[e] = sum;
        }
    }
    if (!SINGLE && tid == 0) a.counted[blockIdx.x] = counted;
    __syncthreads();
    if (SINGLE) {
        scan_experts<THREADS>(total, first, E, warps);
        for (int e = tid; e <= E; e += THREADS) {
            a.offsets[e] = first[e];
            if (e < E && a.counts) a.counts[e] = total[e];
        }
    }
    if (l < k) {
        constexpr int U = 8;  // tokens read at once
        place = (uint32_t)(t0 * k) + l;
        for (int i = 0; i < min(n_here, kept_tokens); i++, place += k) {
            const int32_t c = kept[(i * NG + run) * k + l];
            const int32_t at = c < 0 ? -1 : (c >> 10) + mine[c & 1023] + (SINGLE ? first[c & 1023] : 0);
            a.position[place] = at;
            if (SINGLE && c >= 0) a.token[at] = (int32_t)(t0 + i);
        }
        for (int i0 = kept_tokens; i0 < n_here; i0 += U, place += U * k) {
            int32_t e[U], at[U];
#pragma unroll
            for (int i = 0; i < U; i++) {
                const bool ok = i0 + i < n_here;
                e[i] = ok ? a.expert[place + i * k] : -1;
                at[i] = ok ? a.position[place + i * k] : -1;
            }
#pragma unroll
            for (int i = 0; i < U; i++) {
                if (e[i] < 0) continue;
                at[i] += mine[e[i]] + (SINGLE ? first[e[i]] : 0);
                a.position[place + i * k] = at[i];
                if (SINGLE) a.token[at[i]] = (int32_t)(t0 + i0 + i);
            }
        }
    }
    if (!(SINGLE ? (void *)a.slope : (void *)a.psum)) return;
    __syncthreads();
    float *pf = reinterpret_cast<float *>(cnt);
#pragma unroll
    for (int s = 0; s < S; s++)
        if (l * S + s < E && run < runs) pf[run * E + l * S + s] = s & 1 ? ps[s / 2].y : ps[s / 2].x;
    __syncthreads();
    float *psum = SINGLE ? reinterpret_cast<float *>(first) : a.psum + (int)blockIdx.x * E;  // first's rows are done with
    if (G == 32) {
        for (int e = tid; e < E; e += THREADS) {
            float sum = 0.0f;
#pragma unroll 8
            for (int g = 0; g < runs; g++) sum += pf[g * E + e];
            psum[e] = sum;
        }
    } else {
        for (int e = tid >> 5; e < E; e += THREADS / 32) {
            float sum = 0.0f;
            for (int g = lane; g < runs; g += 32) sum += pf[g * E + e];
            sum = group_sum<32>(sum);
            if (lane == 0) psum[e] = sum;
        }
    }
    if (SINGLE) {
        __syncthreads();
        balance<THREADS>(a, total, psum, counted, first[E], reinterpret_cast<float *>(warps));
    }
}

// The rows of every tile: CTA i adds up the counts of the tiles before its own and of all tiles, and the
// experts' first rows; its tokens' ranks become rows.  The CTA behind the last tile makes the loss.
// Bound: latency (152 tiles' counts of 256 experts, 156 KB from L2 a CTA, then two dependent accesses).
__global__ void __launch_bounds__(1024) route_rows_kernel(const RouteArgs a, int tiles, int64_t tile_tokens) {
    __shared__ int4 part_b[1024], part_n[1024];
    __shared__ int32_t before[1024], total[1024], first[1025], warps[32], counted;
    pdl_wait();
    pdl_trigger();
    const int E = a.experts, tid = threadIdx.x, tile = blockIdx.x;
    int wide = 8;  // threads across the experts, four each; the rest share out the tiles
    while (4 * wide < E) wide *= 2;
    const int parts = min(1024 / wide, 32), part = tid / wide, e = 4 * (tid % wide);
    int4 b = make_int4(0, 0, 0, 0), n = b;
    float4 p = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
    const bool vec = E % 4 == 0;
    const auto four = [&](const int32_t *at) {  // four experts' figures, zeros behind the last
        if (vec) return *reinterpret_cast<const int4 *>(at);
        return make_int4(at[0], e + 1 < E ? at[1] : 0, e + 2 < E ? at[2] : 0, e + 3 < E ? at[3] : 0);
    };
    const int64_t lo = tile * tile_tokens * a.k, hi = min((tile + 1) * tile_tokens, a.tokens) * a.k;
    constexpr int U = 2;
    int32_t x[U], at[U];
    const auto load = [&](int64_t i0) {  // U choices a thread and the ranks in their tile
#pragma unroll
        for (int u = 0; u < U; u++) {
            const int64_t i = i0 + 1024 * u;
            x[u] = i < hi ? a.expert[i] : -1;
            at[u] = i < hi ? a.position[i] : -1;
        }
    };
    load(lo + tid);  // the first ones while the tiles' counts add up
    const bool loss = tile == tiles;  // all tiles' sums of p in the place of the counts before
    if (tid == 0) counted = 0;
    const int32_t own = loss && tid < tiles ? a.counted[tid] : 0;
    if (e < E && part < parts) {
        if (loss) {
#pragma unroll 5
            for (int i = part; i < tiles; i += parts) {
                const int4 c = four(a.hist + i * E + e), d = four(reinterpret_cast<const int32_t *>(a.psum) + i * E + e);
                n.x += c.x, n.y += c.y, n.z += c.z, n.w += c.w;
                p.x += __int_as_float(d.x), p.y += __int_as_float(d.y), p.z += __int_as_float(d.z), p.w += __int_as_float(d.w);
            }
            b = make_int4(__float_as_int(p.x), __float_as_int(p.y), __float_as_int(p.z), __float_as_int(p.w));
        } else {
#pragma unroll 10
            for (int i = part; i < tiles; i += parts) {
                const int4 c = four(a.hist + i * E + e);
                n.x += c.x, n.y += c.y, n.z += c.z, n.w += c.w;
                if (i < tile) b.x += c.x, b.y += c.y, b.z += c.z, b.w += c.w;
            }
        }
    }
    // [part][expert], so that a thread per expert reads one line of banks
    part_b[tid] = b, part_n[tid] = n;
    __syncthreads();
    if (own) atomicAdd(&counted, own);
    if (tid < E) {
        const int32_t *pb = reinterpret_cast<const int32_t *>(part_b) + tid, *pn = reinterpret_cast<const int32_t *>(part_n) + tid;
        int32_t sb = 0, sn = 0;
        float sp = 0.0f;
#pragma unroll 4
        for (int q = 0; q < parts; q++) {
            sn += pn[4 * wide * q];
            if (loss) sp += __int_as_float(pb[4 * wide * q]);
            else sb += pb[4 * wide * q];
        }
        before[tid] = loss ? __float_as_int(sp) : sb, total[tid] = sn;
    }
    __syncthreads();
    scan_experts<1024>(total, first, E, warps);
    if (loss) {
        balance<1024>(a, total, reinterpret_cast<const float *>(before), counted, first[E], reinterpret_cast<float *>(warps));
        return;
    }
    if (tile == 0) {
        if (tid < E) {
            a.offsets[tid] = first[tid];
            if (a.counts) a.counts[tid] = total[tid];
        }
        if (tid == 0) a.offsets[E] = first[E];
    }
    if (tid < E) before[tid] += first[tid];
    __syncthreads();
    for (int64_t i0 = lo + tid; i0 < hi; i0 += 1024 * U) {
#pragma unroll
        for (int u = 0; u < U; u++) {
            const int64_t i = i0 + 1024 * u;
            if (x[u] < 0) continue;
            at[u] += before[x[u]];
            a.position[i] = at[u];
            a.token[at[u]] = (int32_t)((uint32_t)i / (uint32_t)a.k);
        }
        load(i0 + 1024 * U);
    }
}

// G lanes a token; the chosen experts' extra gradient reaches its lanes through shared memory, a row
// of zeros per group of lanes that is cleared again.  The grid is what is resident (eight CTAs an SM: 12.8 us for 9.8).
// 32768 tokens of 256 experts in bf16, 8 choices: 10 us, 3.4 TB/s; bound: the issue slots (65% in use, about 230
// instructions a token).
constexpr int bwd_ctas(int S) { return S <= 2 ? 5 : S == 4 ? 4 : S <= 16 ? 3 : 2; }  // of an SM: as many as its registers hold
template <int XKIND, int G, int S>
__global__ void __launch_bounds__(256, bwd_ctas(S)) route_bwd_kernel(const RouteArgs a, const float *dweight, const float *dloss,
                                                        void *dlogits) {
    constexpr int NG = 256 / G, ESZ = XKIND == FP8DL_BF16 ? 2 : 4;
    __shared__ __align__(8) float extra[NG][G * S];
    const int E = a.experts, k = a.k, lane = threadIdx.x & 31, run = threadIdx.x / G, l = threadIdx.x % G, i0 = l * S;
    float *mine = extra[run];
#pragma unroll
    for (int s = 0; s < S; s++) mine[i0 + s] = 0.0f;
    pdl_wait();
    pdl_trigger();
    const float dl = dloss ? *dloss : 0.0f;
    constexpr int PAIRS = Logits<XKIND, S>::PAIRS;
    float2 even[PAIRS];
#pragma unroll
    for (int p = 0; p < PAIRS; p++)
        even[p] = make_float2(dloss && i0 + 2 * p < E ? dl * a.slope[i0 + 2 * p] : 0.0f,
                              dloss && 2 * p + 1 < S && i0 + 2 * p + 1 < E ? dl * a.slope[i0 + 2 * p + 1] : 0.0f);
    // less their mean, which drops out of dp - <p, dp>: with experts used evenly little is left to cancel
    float2 mean2 = f2(0.0f);
#pragma unroll
    for (int p = 0; p < PAIRS; p++) mean2 = __fadd2_rn(mean2, even[p]);
    const float mean = group_sum<G>(mean2.x + mean2.y) / (float)E;
#pragma unroll
    for (int p = 0; p < PAIRS; p++)  // zeros stay behind the last expert, where p is zero
        even[p] = make_float2(i0 + 2 * p < E ? even[p].x - mean : 0.0f, i0 + 2 * p + 1 < E ? even[p].y - mean : 0.0f);
    __syncwarp();
    const uint32_t gmask = G == 32 ? 0xffffffffu : ((1u << (G & 31)) - 1u) << (lane & ~(G - 1));
    const int64_t step = (int64_t)gridDim.x * NG, rounds = (a.tokens + step - 1) / step;
    int32_t pick_next;
    float w_next, dw_next;
    Logits<XKIND, S> x_next;
    const auto load = [&](int64_t r) {  // of the group's token in round r
        const int64_t t = r * step + (int64_t)blockIdx.x * NG + run;
        const bool here = r < rounds && t < a.tokens;
        pick_next = -1;
        w_next = dw_next = 0.0f;
        if (here && l < k) {
            pick_next = a.expert[t * k + l];
            w_next = a.weight[t * k + l];
            if (dweight) dw_next = dweight[t * k + l];
        }
        if (here) x_next.load(static_cast<const char *>(a.logits) + (t * E + i0) * ESZ, E, i0, a.vec);
        else x_next.none();
    };
    load(0);
    for (int64_t r = 0; r < rounds; r++) {
        const int64_t t = r * step + (int64_t)blockIdx.x * NG + run;
        const bool here = t < a.tokens;
        const int32_t pick = pick_next < E ? pick_next : -1;
        const float w = pick >= 0 ? w_next : 0.0f, dw = pick >= 0 ? dw_next : 0.0f;
        const Logits<XKIND, S> x = x_next;
        if (S < 16) load(r + 1);  // under way meanwhile
        const bool some = __shfl_sync(0xffffffffu, pick, lane & ~(G - 1)) >= 0;
        float m = rt::NEG_INF;
#pragma unroll
        for (int p = 0; p < PAIRS; p++) m = fmaxf(m, fmaxf(x.pair(p).x, x.pair(p).y));  // NaN does not count, as in the choice
        m = group_max(m, gmask);
        if (!some) m = 0.0f;
        float2 v[PAIRS], z2 = f2(0.0f), even2 = f2(0.0f);
#pragma unroll
        for (int p = 0; p < PAIRS; p++) {
            v[p] = route_exp2(x.pair(p), m);
            z2 = __fadd2_rn(z2, v[p]);
            even2 = __ffma2_rn(v[p], even[p], even2);
        }
        // three sums at once: of the exponentials, of theirs times the loss's slopes, and <dw, w>
        float z = z2.x + z2.y, loss = even2.x + even2.y, dot = dw * w;
#pragma unroll
        for (int o = G / 2; o > 0; o >>= 1) {
            z += __shfl_xor_sync(0xffffffffu, z, o);
            loss += __shfl_xor_sync(0xffffffffu, loss, o);
            dot += __shfl_xor_sync(0xffffffffu, dot, o);
        }
        const float inv = some ? __frcp_rn(z) : 0.0f;
        // the chosen experts' part of <p, dp> is <dw, w>, and with `normalize` nothing: their weights add up to 1.  The first
        // choice's weight is then 1 / (sum of the chosen exponentials)
        float d = dw;
        if (a.normalize) d = (dw - dot) * (z * __shfl_sync(0xffffffffu, w, lane & ~(G - 1)));
        const float all = fmaf(dot, a.normalize ? 0.0f : 1.0f, loss * inv);
        if (pick >= 0) mine[pick] = d;
        __syncwarp();
#pragma unroll
        for (int p = 0; p < PAIRS; p++) {
            const float2 extra2 = S > 1 ? *reinterpret_cast<const float2 *>(mine + i0 + 2 * p) : make_float2(mine[i0], 0.0f);
            v[p] = __fmul2_rn(__fmul2_rn(v[p], f2(inv)), __fadd2_rn(__fadd2_rn(even[p], extra2), f2(-all)));
            if (!some) v[p] = f2(0.0f);
        }
        __syncwarp();
        if (pick >= 0) mine[pick] = 0.0f;
        if (here && i0 < E) {
            char *to = static_cast<char *>(dlogits) + (t * E + i0) * ESZ;
            if (a.vec && S * ESZ >= 4) {
                constexpr int WORDS = Logits<XKIND, S>::WORDS;
                uint32_t u[WORDS];
#pragma unroll
                for (int p = 0; p < PAIRS; p++) {
                    if (XKIND == FP8DL_BF16) {
                        const __nv_bfloat162 h = __floats2bfloat162_rn(v[p].x, v[p].y);
                        u[p < WORDS ? p : 0] = *reinterpret_cast<const uint32_t *>(&h);
                    } else {
                        u[2 * p < WORDS ? 2 * p : 0] = __float_as_uint(v[p].x);
                        if (S > 1) u[2 * p + 1 < WORDS ? 2 * p + 1 : 0] = __float_as_uint(v[p].y);
                    }
                }
                if constexpr (S * ESZ >= 16) {
#pragma unroll
                    for (int q = 0; q < S * ESZ / 16; q++)
                        *reinterpret_cast<uint4 *>(to + 16 * q) = make_uint4(u[4 * q], u[4 * q + 1], u[4 * q + 2], u[4 * q + 3]);
                } else if constexpr (S * ESZ == 8) {
                    *reinterpret_cast<uint2 *>(to) = make_uint2(u[0], u[1]);
                } else {
                    *reinterpret_cast<uint32_t *>(to) = u[0];
                }
            } else {
#pragma unroll
                for (int s = 0; s < S; s++) {
                    const float y = s & 1 ? v[s / 2].y : v[s / 2].x;
                    if (i0 + s >= E) continue;
                    if (XKIND == FP8DL_BF16) reinterpret_cast<__nv_bfloat16 *>(to)[s] = __float2bfloat16_rn(y);
                    else reinterpret_cast<float *>(to)[s] = y;
                }
            }
        }
        __syncwarp();
        if (S >= 16) load(r + 1);
    }
}

// Lanes of a token and experts of a lane, for n experts: the fewest lanes that hold them one each, 32 lanes
// from 17 experts on.
static void route_shape(int n, int &g, int &s) {
    g = n <= 8 ? 8 : n <= 16 ? 16 : 32;
    s = 1;
    while (g * s < n) s *= 2;
}

// Whether the lanes' S logits are whole aligned words of a row (the rows start on 16 bytes then, or on
// a word of the lane's size).
static bool route_vec(int n, int s, int esz) { return n % s == 0 && ((int64_t)n * esz) % (s * esz < 16 ? s * esz : 16) == 0; }

template <int XKIND, int G, int S>
static fp8dl_status launch_route(const RouteArgs &a, int tiles, int64_t tile_tokens, int dev, cudaStream_t st, bool pdl) {
    constexpr int THREADS = S >= 16 ? 512 : 1024;
    constexpr int NG = THREADS / G;
    const size_t smem = (size_t)NG * (a.experts + (a.per < rt::KEPT ? a.per : rt::KEPT) * a.k) * 4;
    const bool single = tiles == 1;
    auto *kernel = single ? route_kernel<XKIND, G, S, THREADS, true> : route_kernel<XKIND, G, S, THREADS, false>;
    constexpr size_t most = (size_t)NG * (G * S + rt::KEPT * (G < rt::MAX_K ? G : rt::MAX_K)) * 4;  // with the static arrays past 48 KB
    static std::atomic<uint64_t> done[2];
    FP8DL_TRY(allow_smem(kernel, most, dev, done[single], "moe_route"));
    (void)launch_kernel(kernel, dim3((unsigned)tiles), dim3(THREADS), smem, st, 0, pdl, a);
    note_launch();
    FP8DL_TRY(check_launch("moe_route"));
    if (single) return FP8DL_OK;
    (void)launch_kernel(route_rows_kernel, dim3((unsigned)(tiles + (a.slope ? 1 : 0))), dim3(1024), 0, st, 0, pdl, a, tiles,
                        tile_tokens);
    note_launch();
    return check_launch("moe_route(rows)");
}

template <int XKIND, int G, int S>
static void launch_route_bwd(const RouteArgs &a, const float *dweight, const float *dloss, void *dlogits, int sms,
                             cudaStream_t st, bool pdl) {
    const int64_t ctas = (a.tokens + 256 / G - 1) / (256 / G), most = (int64_t)sms * bwd_ctas(S);
    (void)launch_kernel(route_bwd_kernel<XKIND, G, S>, dim3((unsigned)(ctas < most ? ctas : most)), dim3(256), 0, st, 0, pdl, a,
                        dweight, dloss, dlogits);
    note_launch();
}

static fp8dl_status check_route(const void *logits, int32_t dtype, int64_t tokens, int32_t n_experts, int32_t k) {
    FP8DL_CHECK_ARG(dtype == FP8DL_F32 || dtype == FP8DL_BF16, "dtype must be FP8DL_F32 or FP8DL_BF16");
    FP8DL_CHECK_ARG(n_experts >= 1 && n_experts <= kMaxGroups, "n_experts must be in [1, %d]", kMaxGroups);
    FP8DL_CHECK_ARG(k >= 1 && k <= rt::MAX_K && k <= n_experts, "k must be in [1, min(n_experts, %d)]", rt::MAX_K);
    if (tokens < 0 || tokens >= (int64_t(1) << 31) || tokens * k >= (int64_t(1) << 31))
        return fail(FP8DL_ERR_SHAPE, "tokens (%lld) must not be negative and tokens * k must be below 2^31", (long long)tokens);
    FP8DL_CHECK_ARG(tokens == 0 || logits, "logits is NULL");
    return FP8DL_OK;
}

}  // namespace fp8dl

using namespace fp8dl;

extern "C" size_t moe_route_workspace_size(int64_t tokens, int32_t n_experts) {
    if (tokens <= 0 || n_experts < 1 || n_experts > kMaxGroups) return 0;
    const size_t tiles = tokens < rt::MAX_TILES ? (size_t)tokens : rt::MAX_TILES;
    return (tiles * n_experts + 3) / 4 * 16 + (tiles + 3) / 4 * 16 + tiles * n_experts * 4;
}

extern "C" fp8dl_status moe_route(const void *logits, int32_t dtype, int64_t tokens, int32_t n_experts, int32_t k,
                                  const uint8_t *valid, int32_t normalize, int32_t *expert, float *weight,
                                  int32_t *position, int32_t *token, int32_t *offsets, int32_t *counts, float *slope,
                                  float *loss, void *workspace, size_t workspace_bytes, fp8dl_stream_t stream) {
    FP8DL_NVTX("moe_route");
    FP8DL_TRY(check_route(logits, dtype, tokens, n_experts, k));
    FP8DL_CHECK_ARG(offsets && (tokens == 0 || (expert && weight && position && token)),
                    "expert, weight, position, token and offsets must be non-NULL");
    FP8DL_CHECK_ARG(!slope == !loss, "slope and loss come together");
    if (!aligned16(logits)) return fail(FP8DL_ERR_ALIGN, "logits must be 16-byte aligned");
    if (!aligned4(expert) || !aligned4(weight) || !aligned4(position) || !aligned4(token) || !aligned4(offsets) ||
        !aligned4(counts) || !aligned4(slope) || !aligned4(loss))
        return fail(FP8DL_ERR_ALIGN, "expert, weight, position, token, offsets, counts, slope and loss must be 4-byte aligned");
    if (tokens > 0) {
        if (!workspace || workspace_bytes < moe_route_workspace_size(tokens, n_experts))
            return fail(FP8DL_ERR_WORKSPACE, "moe_route needs a workspace of %zu bytes (got %zu)",
                        moe_route_workspace_size(tokens, n_experts), workspace ? workspace_bytes : (size_t)0);
        if (!aligned16(workspace)) return fail(FP8DL_ERR_ALIGN, "workspace must be 16-byte aligned");
    }
    int dev = 0, sms = 0;
    FP8DL_TRY(current_device(&dev, &sms));
    cudaStream_t st = (cudaStream_t)stream;
    if (tokens == 0) {
        if (cudaMemsetAsync(offsets, 0, (size_t)(n_experts + 1) * 4, st) != cudaSuccess ||
            (counts && cudaMemsetAsync(counts, 0, (size_t)n_experts * 4, st) != cudaSuccess) ||
            (slope && cudaMemsetAsync(slope, 0, (size_t)n_experts * 4, st) != cudaSuccess) ||
            (loss && cudaMemsetAsync(loss, 0, 4, st) != cudaSuccess))
            return check_launch("moe_route(empty)");
        return FP8DL_OK;
    }
    int g, s;
    route_shape(n_experts, g, s);
    const int esz = dtype == FP8DL_BF16 ? 2 : 4, runs = (s >= 16 ? 512 : 1024) / g;
    const int64_t most = sms < rt::MAX_TILES ? sms : rt::MAX_TILES;
    RouteArgs a = {};
    a.logits = logits;
    a.tokens = tokens;
    a.experts = n_experts;
    a.k = k;
    a.normalize = normalize != 0;
    a.vec = route_vec(n_experts, s, esz);
    a.valid = valid;
    a.expert = expert, a.position = position, a.token = token, a.offsets = offsets, a.counts = counts;
    a.weight = weight, a.slope = slope, a.loss = loss;
    // few tokens: one CTA and one launch, up to two tokens a run (64 tokens of 64 experts 4.8 us against 5.6, 256 of 8
    // 5.6 against 6.3; with four 7.2 against 5.7, 8.4 against 6.3)
    a.per = tokens <= 2 * runs ? (tokens + runs - 1) / runs : (tokens + most * runs - 1) / (most * runs);
    const int64_t tile_tokens = a.per * runs;
    const int tiles = (int)((tokens + tile_tokens - 1) / tile_tokens);
    a.hist = static_cast<int32_t *>(workspace);
    a.counted = a.hist + (tiles * n_experts + 3) / 4 * 4;
    a.psum = slope ? reinterpret_cast<float *>(a.counted + (tiles + 3) / 4 * 4) : nullptr;
    const bool pdl = short_call_bytes((double)tokens * n_experts * esz);
    fp8dl_status r = FP8DL_OK;
#define FP8DL_ROUTE(g_, s_)                                                                          \
    r = dtype == FP8DL_BF16 ? launch_route<FP8DL_BF16, g_, s_>(a, tiles, tile_tokens, dev, st, pdl)  \
                            : launch_route<FP8DL_F32, g_, s_>(a, tiles, tile_tokens, dev, st, pdl)
    if (g == 8) FP8DL_ROUTE(8, 1);
    else if (g == 16) FP8DL_ROUTE(16, 1);
    else if (s == 1) FP8DL_ROUTE(32, 1);
    else if (s == 2) FP8DL_ROUTE(32, 2);
    else if (s == 4) FP8DL_ROUTE(32, 4);
    else if (s == 8) FP8DL_ROUTE(32, 8);
    else if (s == 16) FP8DL_ROUTE(32, 16);
    else FP8DL_ROUTE(32, 32);
#undef FP8DL_ROUTE
    return r;
}

extern "C" fp8dl_status moe_route_bwd(const void *logits, int32_t dtype, int64_t tokens, int32_t n_experts, int32_t k,
                                      int32_t normalize, const int32_t *expert, const float *weight,
                                      const float *dweight, const float *slope, const float *dloss, void *dlogits,
                                      fp8dl_stream_t stream) {
    FP8DL_NVTX("moe_route_bwd");
    FP8DL_TRY(check_route(logits, dtype, tokens, n_experts, k));
    FP8DL_CHECK_ARG(tokens == 0 || (expert && weight && dlogits), "expert, weight and dlogits must be non-NULL");
    FP8DL_CHECK_ARG(tokens == 0 || !dloss || slope, "dloss without slope");
    if (!aligned16(logits) || !aligned16(dlogits)) return fail(FP8DL_ERR_ALIGN, "logits and dlogits must be 16-byte aligned");
    if (!aligned4(expert) || !aligned4(weight) || !aligned4(dweight) || !aligned4(slope) || !aligned4(dloss))
        return fail(FP8DL_ERR_ALIGN, "expert, weight, dweight, slope and dloss must be 4-byte aligned");
    int sms = 0;
    FP8DL_TRY(current_device(nullptr, &sms));
    if (tokens == 0) return FP8DL_OK;
    // lanes of a token (a choice each) and experts of a lane: the fewest lanes that hold them eight each (16384 tokens of 64:
    // 4.4 us, with 32 lanes of two 5.3; 16 lanes of 16 are slower than 32 of eight: 32768 of 256 11.6 against 9.8)
    const int g = n_experts <= 64 && k <= 8 ? 8 : n_experts <= 128 && k <= 16 ? 16 : 32;
    int s = 1;
    while (g * s < n_experts) s *= 2;
    RouteArgs a = {};
    a.logits = logits;
    a.tokens = tokens;
    a.experts = n_experts;
    a.k = k;
    a.normalize = normalize != 0;
    a.vec = route_vec(n_experts, s, dtype == FP8DL_BF16 ? 2 : 4);
    a.expert = const_cast<int32_t *>(expert);
    a.weight = const_cast<float *>(weight);
    a.slope = const_cast<float *>(slope);
    cudaStream_t st = (cudaStream_t)stream;
    const bool pdl = short_call_bytes((double)tokens * n_experts * (dtype == FP8DL_BF16 ? 4.0 : 8.0));
#define FP8DL_ROUTE(g_, s_)                                                                             \
    dtype == FP8DL_BF16 ? launch_route_bwd<FP8DL_BF16, g_, s_>(a, dweight, dloss, dlogits, sms, st, pdl) \
                        : launch_route_bwd<FP8DL_F32, g_, s_>(a, dweight, dloss, dlogits, sms, st, pdl)
#define FP8DL_LANES(g_)                 \
    if (s == 1) FP8DL_ROUTE(g_, 1);      \
    else if (s == 2) FP8DL_ROUTE(g_, 2); \
    else if (s == 4) FP8DL_ROUTE(g_, 4); \
    else if (s == 8) FP8DL_ROUTE(g_, 8)
    if (g == 8) {
        FP8DL_LANES(8);
    } else if (g == 16) {
        FP8DL_LANES(16);
    } else {
        FP8DL_LANES(32);
        else if (s == 16) FP8DL_ROUTE(32, 16);
        else FP8DL_ROUTE(32, 32);
    }
#undef FP8DL_LANES
#undef FP8DL_ROUTE
    return check_launch("moe_route_bwd");
}
