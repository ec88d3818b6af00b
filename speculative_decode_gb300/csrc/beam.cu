// beam.cu -- one step of beam search: the best continuations over a group's
// beams and the vocabulary, and the page tables and tail pages behind them.
//
// Selection. A continuation of beam w by token t has the value
//   score[w] + (x[w][t] - lse_w),   lse_w = log(sum_t exp x[w][t]);
// a finished beam has one, its end token at the beam's score. The K largest
// values of a group win; equal values go to the lower beam, and inside a beam
// to the larger logit, then the lower token. A NaN logit counts as -inf, +inf as the
// largest finite value.
//
// One pass over the logits: a CTA keeps a chunk of a row in registers, and takes
// from it the chunk's maximum, the sum of exp(x - max) and its K largest
// logits (a row's order is its logits' order, so no sum is needed to choose
// them). The last CTA of a group to finish (one atomic counter a group, no
// spinning) merges the sums into each row's lse and the chunks' picks into the
// group's. lse and the values are formed in 64 bits, so that beams are told
// apart down to the accuracy of the sums (about 1e-7).
//
// Choosing K of a chunk: each of the eight warps finds its J-th largest lane
// maximum, J = ceil(K / 8). At least J values of each warp reach the least of
// those, so the K largest of the chunk do; the few values that reach it (about
// 20 for K = 8) are collected and ranked by counting. When more than 128 do
// (constant rows, heavy ties), they are taken one by one as block-wide maxima.
//
// Reordering. Child i of a group continues beam p = parents[i]. Pages that are
// full are shared: the child's table row starts with its parent's. The pages
// from the first unfilled one on belong to one beam alone: the lowest child of
// a parent keeps its parent's, and the k-th other child of the group takes
// those of the k-th beam that has no child (there are as many), into which the
// parent's rows of the unfilled page are copied. Nothing that is read is
// written, so one kernel does it in any order. Bound: bytes copied.
#include <cfloat>
#include <type_traits>

#include "common.cuh"

namespace sa {

namespace {

constexpr int kThreads = 256;
constexpr int kWarps = kThreads / 32;
constexpr int kCap = 1024;       // collected candidates of a chunk
constexpr int kRankMost = 128;   // ranked by counting up to this many
constexpr int kMergeCap = 2048;  // candidates of one merge step
constexpr int kMaxBeams = kMaxBeamWidth;
constexpr int kIndexBits = 27;   // tokens in a merge key
constexpr uint32_t kIndexMask = (1u << kIndexBits) - 1;
constexpr float kLog2e = 1.4426950408889634f;

// Unsigned integers in the order of the floats (-inf lowest, no NaN).
__device__ __forceinline__ uint32_t order32(float x) {
    const uint32_t u = __float_as_uint(x + 0.f);  // -0 becomes +0
    return u ^ (static_cast<uint32_t>(static_cast<int32_t>(u) >> 31) | 0x80000000u);
}

__device__ __forceinline__ float order32_value(uint32_t k) {
    return __uint_as_float(k & 0x80000000u ? k ^ 0x80000000u : ~k);
}

__device__ __forceinline__ uint64_t order64(double x) {
    const long long u = __double_as_longlong(x + 0.0);
    return static_cast<uint64_t>(u) ^ (static_cast<uint64_t>(u >> 63) | 0x8000000000000000ull);
}

__device__ __forceinline__ double order64_value(uint64_t k) {
    return __longlong_as_double(static_cast<long long>(k >> 63 ? k ^ 0x8000000000000000ull : ~k));
}

constexpr uint32_t kOrderNegInf = 0x007fffffu;  // order32(-inf)

// A chunk's candidates as keys: larger logit first, then lower token. 0: none.
__device__ __forceinline__ uint64_t pick_key(float x, int idx) {
    return static_cast<uint64_t>(order32(x)) << 32 | ~static_cast<uint32_t>(idx);
}

// Largest key of a warp.
__device__ __forceinline__ uint64_t warp_max(uint64_t k) {
    const uint32_t hi = static_cast<uint32_t>(k >> 32);
    const uint32_t top = __reduce_max_sync(0xffffffffu, hi);
    const uint32_t lo = __reduce_max_sync(0xffffffffu, hi == top ? static_cast<uint32_t>(k) : 0u);
    return static_cast<uint64_t>(top) << 32 | lo;
}

struct Logits32 {
    using type = float;
    static constexpr int kVec = 4;
    static __device__ __forceinline__ float one(const float *p) { return *p; }
    static __device__ __forceinline__ void vec(const float *p, float *x) {
        const float4 v = __ldcs(reinterpret_cast<const float4 *>(p));
        x[0] = v.x;
        x[1] = v.y;
        x[2] = v.z;
        x[3] = v.w;
    }
};

struct Logits16 {
    using type = uint16_t;
    static constexpr int kVec = 8;
    static __device__ __forceinline__ float one(const uint16_t *p) {
        return __uint_as_float(static_cast<uint32_t>(*p) << 16);
    }
    static __device__ __forceinline__ void vec(const uint16_t *p, float *x) {
        const uint4 v = __ldcs(reinterpret_cast<const uint4 *>(p));
        const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            x[2 * i] = bf16_lo(w[i]);
            x[2 * i + 1] = bf16_hi(w[i]);
        }
    }
};

// A merge candidate: value first, then beam, logit and token.
struct Candidate {
    uint64_t value;  // order64 of the value; 0: none
    uint64_t rest;   // (31 - beam) : 5, order32(logit) : 32, inverted token : 27
};

__device__ __forceinline__ bool before(const Candidate &a, const Candidate &b) {
    return a.value > b.value || (a.value == b.value && a.rest > b.rest);
}

__device__ __forceinline__ Candidate make_candidate(double value, int beam, uint32_t logit_order, uint32_t token) {
    if (!(value > -INFINITY)) return Candidate{0, 0};
    return Candidate{order64(value), static_cast<uint64_t>(kMaxBeams - 1 - beam) << 59 |
                                         static_cast<uint64_t>(logit_order) << kIndexBits | (kIndexMask - token)};
}

struct SelectShared {
    float m[kWarps], s[kWarps];
    uint64_t tau[kWarps];
    int n, last;
    uint64_t red[2][kWarps];
    // merge
    double lse[kMaxBeams];
    float row_m[kMaxBeams];
    double row_s[kMaxBeams];
    Candidate cred[2][kWarps];
    Candidate best[kMaxBeams];
    int32_t out_token[kMaxBeams], out_beam[kMaxBeams];
    float out_score[kMaxBeams];
    union {
        uint64_t keys[kCap];
        Candidate cand[kMergeCap];
    };
    Candidate kept[kRankMost];
};

// The K largest of the n candidates in S.cand to S.best, sorted (none: value
// 0); returns how many there are. Called by the whole block.
__device__ int merge_best(SelectShared &S, int n, int K) {
    const int t = threadIdx.x, lane = t & 31, warp = t >> 5;
    // threshold on the values' upper halves: the least of the warps' J-th
    // largest lane maxima (as in a chunk)
    uint32_t top = 0;
    for (int e = t; e < n; e += kThreads) top = max(top, static_cast<uint32_t>(S.cand[e].value >> 32));
    const int J = (K + kWarps - 1) / kWarps;
    uint32_t jth = 0;
    for (int j = 0; j < J; ++j) {
        jth = __reduce_max_sync(0xffffffffu, top);
        const uint32_t who = __ballot_sync(0xffffffffu, top == jth);
        if (lane == __ffs(who) - 1) top = 0;
    }
    if (lane == 0) S.tau[warp] = jth;
    if (t == 0) S.n = 0;
    __syncthreads();
    uint64_t tau = S.tau[0];
#pragma unroll
    for (int w = 1; w < kWarps; ++w) tau = min(tau, S.tau[w]);
    for (int e = t; e < n; e += kThreads) {
        const Candidate c = S.cand[e];
        if (c.value != 0 && (c.value >> 32) >= tau) {
            const int at = atomicAdd(&S.n, 1);
            if (at < kRankMost) S.kept[at] = c;
        }
    }
    __syncthreads();
    const int got = S.n;
    if (got <= kRankMost) {
        if (t < got) {
            const Candidate c = S.kept[t];
            int rank = 0;
            for (int o = 0; o < got; ++o) rank += before(S.kept[o], c);
            if (rank < K) S.best[rank] = c;
        }
        __syncthreads();
        return min(got, K);
    }
    Candidate last{~0ull, ~0ull};
    for (int k = 0; k < K; ++k) {
        Candidate c{0, 0};
        for (int e = t; e < n; e += kThreads) {
            const Candidate x = S.cand[e];
            if (before(last, x) && before(x, c)) c = x;
        }
#pragma unroll
        for (int o = 16; o >= 1; o >>= 1) {
            const Candidate x{__shfl_xor_sync(0xffffffffu, c.value, o), __shfl_xor_sync(0xffffffffu, c.rest, o)};
            if (before(x, c)) c = x;
        }
        if (lane == 0) S.cred[k & 1][warp] = c;
        __syncthreads();
        last = S.cred[k & 1][0];
#pragma unroll
        for (int w = 1; w < kWarps; ++w)
            if (before(S.cred[k & 1][w], last)) last = S.cred[k & 1][w];
        if (t == 0) S.best[k] = last;
    }
    __syncthreads();
    return K;  // more than K candidates have a value
}

// The slots behind the `n` continuations of a value above -inf: continuations
// of value -inf, by beam, larger logit and lower token. One warp; rare (fewer
// than K tokens of the group have any probability).
template <typename L>
__device__ void fill_rest(SelectShared &S, const SelectParams &P, int g, int n) {
    using T = typename L::type;
    const int lane = threadIdx.x & 31;
    for (int w = 0; w < P.W && n < P.K; ++w) {
        const int64_t row = static_cast<int64_t>(g) * P.W + w;
        const bool live = P.scores[row] > -INFINITY;
        const bool done = P.finished != nullptr && P.finished[row] != 0;
        auto put = [&](int token) {
            if (lane == 0) {
                S.out_token[n] = token;
                S.out_beam[n] = w;
                S.out_score[n] = -INFINITY;
            }
            ++n;
        };
        if (done && !live) put(P.eos);
        if (!done && !live) {  // the row's listed logits in their order
            const uint64_t *keys = P.part_keys + row * P.n_chunks * P.K;
            uint64_t last = ~0ull;
            while (n < P.K) {
                uint64_t k = 0;
                for (int e = lane; e < P.n_chunks * P.K; e += 32) {
                    const uint64_t x = __ldcg(keys + e);
                    if (x < last && x > k) k = x;
                }
                k = warp_max(k);
                if (k == 0) break;
                put(static_cast<int>(~static_cast<uint32_t>(k)));
                last = k;
            }
        }
        // tokens without probability, in order (of a finished beam: all but its end token)
        const T *x = static_cast<const T *>(P.logits) + row * P.stride;
        for (int t0 = 0; t0 < P.V && n < P.K; t0 += 32) {
            const int t = t0 + lane;
            const bool none = t < P.V && (done ? t != P.eos : !(L::one(x + t) > -INFINITY));
            uint32_t who = __ballot_sync(0xffffffffu, none);
            while (who != 0 && n < P.K) {
                put(t0 + __ffs(who) - 1);
                who &= who - 1;
            }
        }
    }
}

// The last CTA of group g: every row's lse, then the K best of all listed
// candidates.
template <typename L>
__device__ void merge_group(SelectShared &S, const SelectParams &P, int g) {
    const int t = threadIdx.x, lane = t & 31, warp = t >> 5;
    const int64_t row0 = static_cast<int64_t>(g) * P.W;
    for (int w = warp; w < P.W; w += kWarps) {
        const float2 *part = P.part_sums + (row0 + w) * P.n_chunks;
        float m = -INFINITY;
        for (int c = lane; c < P.n_chunks; c += 32) m = fmaxf(m, __ldcg(part + c).x);
#pragma unroll
        for (int o = 16; o >= 1; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
        double s = 0.0;
        for (int c = lane; c < P.n_chunks; c += 32) {
            const float2 q = __ldcg(part + c);
            if (q.x > -INFINITY) s += static_cast<double>(q.y) * static_cast<double>(expf(q.x - m));
        }
#pragma unroll
        for (int o = 16; o >= 1; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
        if (lane == 0) {
            S.row_m[w] = m;
            S.row_s[w] = s;
        }
    }
    __syncthreads();
    if (t < P.W) S.lse[t] = static_cast<double>(S.row_m[t]) + log(S.row_s[t]);
    __syncthreads();

    // candidates in steps of kMergeCap, the best of the steps before kept;
    // consecutive candidates are of different rows, so that each warp sees all
    const int64_t total = static_cast<int64_t>(P.n_chunks) * P.K * P.W;
    int n = 0;
    for (int64_t e0 = 0; e0 < total;) {
        const int take = static_cast<int>(min(total - e0, static_cast<int64_t>(kMergeCap - n)));
        if (t < n) S.cand[t] = S.best[t];
        for (int i = t; i < take; i += kThreads) {
            const int w = static_cast<int>((e0 + i) % P.W), at = static_cast<int>((e0 + i) / P.W);
            const int64_t row = row0 + w;
            const float score = P.scores[row];
            Candidate c{0, 0};
            if (P.finished != nullptr && P.finished[row] != 0) {
                if (at == 0) c = make_candidate(score, w, ~0u, P.eos);
            } else {
                // a rank of all the row's chunks, then the next
                const uint64_t key = __ldcg(P.part_keys + (row * P.n_chunks + at % P.n_chunks) * P.K + at / P.n_chunks);
                if (key != 0) {
                    const uint32_t order = static_cast<uint32_t>(key >> 32);
                    c = make_candidate(score + (static_cast<double>(order32_value(order)) - S.lse[w]), w, order,
                                       ~static_cast<uint32_t>(key));
                }
            }
            S.cand[n + i] = c;
        }
        __syncthreads();
        n = merge_best(S, n + take, P.K);
        e0 += take;
    }
    if (t < n) {
        const Candidate c = S.best[t];
        S.out_beam[t] = kMaxBeams - 1 - static_cast<int>(c.rest >> 59);
        S.out_token[t] = static_cast<int>(kIndexMask - (static_cast<uint32_t>(c.rest) & kIndexMask));
        S.out_score[t] = static_cast<float>(order64_value(c.value));
    }
    if (n < P.K && warp == 0) {
        __syncwarp();
        fill_rest<L>(S, P, g, n);
    }
    __syncthreads();
    int ended = 0;
    if (t < P.K) {
        const int64_t at = static_cast<int64_t>(g) * P.K + t;
        const int token = S.out_token[t], beam = S.out_beam[t];
        ended = token == P.eos || (P.finished != nullptr && P.finished[row0 + beam] != 0);
        P.tokens[at] = token;
        P.parents[at] = beam;
    }
    __syncthreads();  // the outputs may be the inputs' buffers
    if (t < P.K) {
        const int64_t at = static_cast<int64_t>(g) * P.K + t;
        P.scores_out[at] = S.out_score[t];
        if (P.finished_out != nullptr) P.finished_out[at] = ended;
    }
}

// E values of a row per thread. kAligned: every row starts on a 16-byte
// boundary and is read in 16-byte groups.
template <typename L, int E, bool kAligned>
__global__ void __launch_bounds__(kThreads) beam_select_kernel(const SelectParams P) {
    using T = typename L::type;
    constexpr int kVec = L::kVec;
    __shared__ SelectShared S;
    const int t = threadIdx.x, lane = t & 31, warp = t >> 5;
    const int64_t row = blockIdx.x / P.n_chunks;
    const int chunk = static_cast<int>(blockIdx.x - row * P.n_chunks);
    const int g = static_cast<int>(row / P.W);

    if (P.finished == nullptr || P.finished[row] == 0) {
        // All rows of a launch are cut alike, whatever their address, so that
        // equal rows have equal sums and equal values.
        const T *x0 = static_cast<const T *>(P.logits) + row * P.stride;
        const int c0 = chunk * P.chunk, c1 = min(P.V, c0 + P.chunk);
        auto index = [&](int e) {
            return c0 + (kAligned ? (t + e / kVec * kThreads) * kVec + e % kVec : t + e * kThreads);
        };
        float x[E];
        if constexpr (kAligned) {
#pragma unroll
            for (int i = 0; i < E / kVec; ++i) {
                const int first = index(i * kVec);
                if (first + kVec <= c1) {
                    L::vec(x0 + first, x + i * kVec);
                } else {
#pragma unroll
                    for (int e = 0; e < kVec; ++e) x[i * kVec + e] = first + e < c1 ? L::one(x0 + first + e) : -INFINITY;
                }
            }
        } else {
#pragma unroll
            for (int e = 0; e < E; ++e) x[e] = index(e) < c1 ? L::one(x0 + index(e)) : -INFINITY;
        }
        // NaN -> -inf, +inf -> largest finite
        float mx = -INFINITY;
#pragma unroll
        for (int e = 0; e < E; ++e) {
            x[e] = fminf(fmaxf(x[e], -INFINITY), FLT_MAX);
            mx = fmaxf(mx, x[e]);
        }
        int at = INT32_MAX;  // the lane maximum's lowest token
#pragma unroll
        for (int e = E - 1; e >= 0; --e) at = x[e] == mx ? index(e) : at;

        uint32_t key = order32(mx);
        const uint32_t wtop = __reduce_max_sync(0xffffffffu, key);
        const float wmax = order32_value(wtop);
        float part[4] = {0.f, 0.f, 0.f, 0.f};
        if (wtop != kOrderNegInf) {
#pragma unroll
            for (int e = 0; e < E; ++e) part[e & 3] += exp2f((x[e] - wmax) * kLog2e);
        }
        float sum = (part[0] + part[1]) + (part[2] + part[3]);
#pragma unroll
        for (int o = 16; o >= 1; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);

        // the warp's J-th largest lane maximum (lower token first among equals)
        const int J = (P.K + kWarps - 1) / kWarps;
        uint64_t jth = 0;
        for (int j = 0; j < J; ++j) {
            const uint32_t top = __reduce_max_sync(0xffffffffu, key);
            if (top <= kOrderNegInf) {
                jth = 0;
                break;
            }
            const uint32_t who = __reduce_min_sync(0xffffffffu, key == top ? static_cast<uint32_t>(at) : ~0u);
            jth = static_cast<uint64_t>(top) << 32 | static_cast<uint32_t>(~who);
            if (key == top && static_cast<uint32_t>(at) == who) key = 0;
        }
        if (lane == 0) {
            S.m[warp] = wmax;
            S.s[warp] = sum;
            S.tau[warp] = jth;
        }
        if (t == 0) S.n = 0;
        __syncthreads();
        uint64_t tau = S.tau[0];
#pragma unroll
        for (int w = 1; w < kWarps; ++w) tau = min(tau, S.tau[w]);
        // tau 0: some warp has too few; every value above -inf is collected
        const float tau_x = tau == 0 ? -INFINITY : order32_value(static_cast<uint32_t>(tau >> 32));
        const int tau_at = tau == 0 ? -1 : static_cast<int>(~static_cast<uint32_t>(tau));
#pragma unroll
        for (int e = 0; e < E; ++e) {
            if (x[e] >= tau_x) {
                if (x[e] > tau_x || index(e) <= tau_at) {
                    const int to = atomicAdd(&S.n, 1);
                    if (to < kCap) S.keys[to] = pick_key(x[e], index(e));
                }
            }
        }
        __syncthreads();
        const int n = S.n;
        uint64_t *out = P.part_keys + (row * P.n_chunks + chunk) * P.K;
        if (n <= kRankMost) {
            for (int k = n + t; k < P.K; k += kThreads) out[k] = 0;
            if (t < n) {
                const uint64_t mine = S.keys[t];
                int rank = 0;
                for (int o = 0; o < n; ++o) rank += S.keys[o] > mine;
                if (rank < P.K) out[rank] = mine;
            }
        } else {
            uint64_t last = ~0ull;
            for (int k = 0; k < P.K; ++k) {
                uint64_t best = 0;
                if (n <= kCap) {
                    for (int o = t; o < n; o += kThreads)
                        if (S.keys[o] < last) best = max(best, S.keys[o]);
                } else {
#pragma unroll
                    for (int e = 0; e < E; ++e) {
                        const uint64_t mine = x[e] > -INFINITY ? pick_key(x[e], index(e)) : 0;
                        if (mine < last) best = max(best, mine);
                    }
                }
                best = warp_max(best);
                if (lane == 0) S.red[k & 1][warp] = best;
                __syncthreads();
                last = S.red[k & 1][0];
#pragma unroll
                for (int w = 1; w < kWarps; ++w) last = max(last, S.red[k & 1][w]);
                if (t == 0) out[k] = last;
            }
        }
        if (t == 0) {
            float m = S.m[0];
            for (int w = 1; w < kWarps; ++w) m = fmaxf(m, S.m[w]);
            float s = 0.f;
            if (m > -INFINITY)
                for (int w = 0; w < kWarps; ++w) s += S.s[w] * exp2f((S.m[w] - m) * kLog2e);
            P.part_sums[row * P.n_chunks + chunk] = make_float2(m, s);
        }
    }

    // ---- count this CTA; the last one of a group merges
    __syncthreads();
    if (t == 0) {
        __threadfence();
        const int prev = atomicAdd(&P.counters[g], 1);
        S.last = prev == P.W * P.n_chunks - 1;
    }
    __syncthreads();
    if (!S.last) return;
    __threadfence();
    merge_group<L>(S, P, g);
    if (t == 0) P.counters[g] = 0;
}

// ------------------------------------------------------------------- reorder
// One CTA per (child, KV head).
__global__ void __launch_bounds__(kThreads) beam_reorder_kernel(const ReorderParams P) {
    const int64_t child = blockIdx.x / P.Hkv;
    const int head = static_cast<int>(blockIdx.x - child * P.Hkv);
    const int lane = threadIdx.x & 31;
    const int64_t row0 = child / P.W * P.W;
    const int i = static_cast<int>(child - row0);
    const bool in = lane < P.W;
    const int p = in ? P.parents[row0 + lane] : 0;
    const int len = in ? P.seq_lens[row0 + lane] : 0;
    const int T = __shfl_sync(0xffffffffu, len, 0);
    const bool odd_parent = __any_sync(0xffffffffu, in && (p < 0 || p >= P.W));
    const int full = T / kPageSize, rem = T % kPageSize;
    const bool odd_len = __any_sync(0xffffffffu, in && len != T) || T < 0 || full + (rem > 0) > P.max_pages;
    if (odd_parent || odd_len) {
        if (threadIdx.x == 0 && i == 0 && head == 0)
            flag_error(P.err, (odd_parent ? kErrBitArg : 0) | (odd_len ? kErrBitQlen : 0));
        return;
    }
    const uint32_t has_child = __reduce_or_sync(0xffffffffu, in ? 1u << p : 0u);
    const uint32_t siblings = __match_any_sync(0xffffffffu, in ? p : kMaxBeams + lane);
    const uint32_t others = __ballot_sync(0xffffffffu, in && lane != __ffs(siblings) - 1);
    const int parent = __shfl_sync(0xffffffffu, p, i);
    const bool moved = others >> i & 1;
    int donor = parent;
    if (moved) {
        uint32_t childless = ~has_child;
        for (int k = __popc(others & ((1u << i) - 1)); k > 0; --k) childless &= childless - 1;
        donor = __ffs(childless) - 1;
    }
    const int32_t *from = P.table + (row0 + parent) * P.max_pages;
    const int32_t *own = P.table + (row0 + donor) * P.max_pages;
    if (head == 0)
        for (int j = threadIdx.x; j < P.max_pages; j += kThreads)
            P.table_out[child * P.max_pages + j] = j < full ? from[j] : own[j];
    if (!moved || rem == 0) return;
    const int src = from[full], dst = own[full];
    if (src < 0 || src >= P.num_pages || dst < 0 || dst >= P.num_pages) {
        if (threadIdx.x == 0) flag_error(P.err, kErrBitPageOOB);
        return;
    }
    const int64_t a = (static_cast<int64_t>(src) * P.Hkv + head) * kPageSize;
    const int64_t b = (static_cast<int64_t>(dst) * P.Hkv + head) * kPageSize;
    const int vecs = rem * (P.row_bytes / 16);
    for (int pool = 0; pool < 2; ++pool) {
        const uint4 *s = reinterpret_cast<const uint4 *>(P.pools[pool] + a * P.row_bytes);
        uint4 *d = reinterpret_cast<uint4 *>(P.pools[pool] + b * P.row_bytes);
        constexpr int kFlight = 8;
        for (int v0 = threadIdx.x; v0 < vecs; v0 += kFlight * kThreads) {
            uint4 r[kFlight];
#pragma unroll
            for (int u = 0; u < kFlight; ++u)
                if (v0 + u * kThreads < vecs) r[u] = __ldcs(s + v0 + u * kThreads);
#pragma unroll
            for (int u = 0; u < kFlight; ++u)
                if (v0 + u * kThreads < vecs) d[v0 + u * kThreads] = r[u];
        }
        if (P.scales[pool] != nullptr)
            for (int k = threadIdx.x; k < rem; k += kThreads) P.scales[pool][b + k] = P.scales[pool][a + k];
    }
}

}  // namespace

int beam_select_chunk_values(bool large) { return kThreads * (large ? 32 : 8); }

cudaError_t launch_beam_select(const SelectParams &p, bool bf16, bool large, bool aligned, cudaStream_t stream) {
    const int64_t ctas = static_cast<int64_t>(p.B) * p.W * p.n_chunks;
    auto pick = [&](auto logits, auto aligned_rows) {
        using L = decltype(logits);
        constexpr bool kAligned = decltype(aligned_rows)::value;
        return large ? beam_select_kernel<L, 32, kAligned> : beam_select_kernel<L, 8, kAligned>;
    };
    using Yes = std::true_type;
    using No = std::false_type;
    auto kernel = bf16 ? (aligned ? pick(Logits16{}, Yes{}) : pick(Logits16{}, No{}))
                       : (aligned ? pick(Logits32{}, Yes{}) : pick(Logits32{}, No{}));
    kernel<<<static_cast<unsigned>(ctas), kThreads, 0, stream>>>(p);
    return cudaGetLastError();
}

cudaError_t launch_beam_reorder(const ReorderParams &p, cudaStream_t stream) {
    beam_reorder_kernel<<<static_cast<unsigned>(p.num_seqs * p.Hkv), kThreads, 0, stream>>>(p);
    return cudaGetLastError();
}

}  // namespace sa
