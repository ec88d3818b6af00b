// rope.cu -- norm and position rotation of query and key heads, on their own
// or on the way into the pages.
//
// A row x is one token's head of 128 values. With a weight w it is first
// normalised, y = x * rsqrt(mean(x^2) + eps) * w; without, y = x. The first R
// values are then rotated: pair j < R/2 is (y[j], y[j + R/2]), or, interleaved,
// (y[2j], y[2j+1]), and (a, b) becomes (a cos t - b sin t, a sin t + b cos t)
// with t = position * inv_freq[j]. Everything is held in 32 bits and rounded
// once at the end (bf16 rows) or quantised from the 32-bit values (int8 and
// int4 page rows). t is formed in 64 bits, as a fraction of a turn: at
// position 10^6 a 32-bit product would be off by up to 0.06 rad.
//
// Half a warp holds a row, a lane eight of its values: four first and four
// second values of pairs where it is rotated, so a rotation stays in the lane.
// With the angles and the weights the row's values A, B of the pairs become
// r (A wc - B ws), r (A ws' + B wc'), four products prepared once a token: about
// 60 instructions a pair of rows, in packed 32-bit arithmetic. A warp takes one
// token, or every `parts`-th group of a token's rows; the next group's loads
// are in flight while one is turned. Bound: bytes moved (a row in, a row out)
// for many tokens, two dependent memory round trips (lengths, then rows) for
// few.
#include <cfloat>

#include "common.cuh"

namespace sa {

namespace {

constexpr int kThreads = 128;
constexpr int kWarps = kThreads / 32;
constexpr int kGroup = 2;  // row pairs of a group: two of queries, or one of keys and one of values

__device__ __forceinline__ float half_warp_sum(float v, uint32_t mask) {
#pragma unroll
    for (int o = 8; o >= 1; o >>= 1) v += __shfl_xor_sync(mask, v, o);
    return v;
}

__device__ __forceinline__ float half_warp_max(float v, uint32_t mask) {
#pragma unroll
    for (int o = 8; o >= 1; o >>= 1) v = fmaxf(v, __shfl_xor_sync(mask, v, o));
    return v;
}

// Two floats in one 64-bit register, and arithmetic on both.
__device__ __forceinline__ uint64_t two(float a, float b) {
    uint64_t d;
    asm("mov.b64 %0, {%1, %2};" : "=l"(d) : "f"(a), "f"(b));
    return d;
}
__device__ __forceinline__ float2 apart(uint64_t v) {
    float2 d;
    asm("mov.b64 {%0, %1}, %2;" : "=f"(d.x), "=f"(d.y) : "l"(v));
    return d;
}
__device__ __forceinline__ uint64_t fma2(uint64_t a, uint64_t b, uint64_t c) {
    uint64_t d;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(d) : "l"(a), "l"(b), "l"(c));
    return d;
}
__device__ __forceinline__ uint64_t mul2(uint64_t a, uint64_t b) {
    uint64_t d;
    asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
    return d;
}

// A lane's eight values of a row: A[0..1] are the first values of its pairs
// (two in each), B[0..1] the second.
struct Eight {
    uint64_t A[2], B[2];
};

template <bool kInterleaved>
__device__ __forceinline__ Eight unpack(uint2 a, uint2 b) {
    if constexpr (kInterleaved)
        return Eight{{two(bf16_lo(a.x), bf16_lo(a.y)), two(bf16_lo(b.x), bf16_lo(b.y))},
                     {two(bf16_hi(a.x), bf16_hi(a.y)), two(bf16_hi(b.x), bf16_hi(b.y))}};
    else
        return Eight{{two(bf16_lo(a.x), bf16_hi(a.x)), two(bf16_lo(a.y), bf16_hi(a.y))},
                     {two(bf16_lo(b.x), bf16_hi(b.x)), two(bf16_lo(b.y), bf16_hi(b.y))}};
}

// Its values as they stand in memory: four at the lane's first place, four at
// its second.
template <bool kInterleaved>
__device__ __forceinline__ void in_order(const Eight &v, float (&y)[8]) {
    const float2 a0 = apart(v.A[0]), a1 = apart(v.A[1]), b0 = apart(v.B[0]), b1 = apart(v.B[1]);
    if constexpr (kInterleaved) {
        y[0] = a0.x, y[1] = b0.x, y[2] = a0.y, y[3] = b0.y;
        y[4] = a1.x, y[5] = b1.x, y[6] = a1.y, y[7] = b1.y;
    } else {
        y[0] = a0.x, y[1] = a0.y, y[2] = a1.x, y[3] = a1.y;
        y[4] = b0.x, y[5] = b0.y, y[6] = b1.x, y[7] = b1.y;
    }
}

// What a lane's values are multiplied with, the row's factor aside: A' = A ac -
// B bs, B' = A as + B bc with the weights in them; a lane that is not rotated
// takes A ac and B bc.
struct Turn {
    uint64_t ac[2], bs[2], as[2], bc[2];  // bs with its sign
};

// The factor rsqrt(mean(x^2) + eps) of the half warp's row. A sum of squares
// past 32 bits is formed again of scaled values (a power of two), so rows of
// any finite values have their norm.
__device__ __forceinline__ float norm_factor(Eight &v, float eps, uint32_t mask) {
    auto squares = [&] {
        uint64_t q = mul2(v.A[0], v.A[0]);
        q = fma2(v.A[1], v.A[1], q);
        q = fma2(v.B[0], v.B[0], q);
        q = fma2(v.B[1], v.B[1], q);
        const float2 p = apart(q);
        return half_warp_sum(p.x + p.y, mask);
    };
    const float ss = squares();
    float r = rsqrtf(fmaf(ss, 1.f / kHeadDim, eps));
    if (!(ss <= FLT_MAX)) {
        const uint64_t down = two(0x1p-70f, 0x1p-70f);
        v = Eight{{mul2(v.A[0], down), mul2(v.A[1], down)}, {mul2(v.B[0], down), mul2(v.B[1], down)}};
        r = rsqrtf(squares() * (1.f / kHeadDim));  // eps is far below such a row's mean
    }
    return r;
}

// The page format of the quantising appends (see kv_append.cu), half a warp a
// row: scale = amax / Cmax and code = round-half-even(y / scale), both by IEEE
// division. The lane's values stand at a .. a + 3 and b .. b + 3.
template <int KB>
__device__ __forceinline__ void store_codes(const float (&y)[8], int l, int a, int b, uint32_t mask, uint8_t *codes,
                                            float *scale) {
    constexpr int kMax = KB == 8 ? 127 : 7;
    float amax = 0.f;
#pragma unroll
    for (int e = 0; e < 8; ++e) amax = fmaxf(amax, fabsf(y[e]));
    amax = half_warp_max(amax, mask);
    const float sc = __fdiv_rn(amax, static_cast<float>(kMax));
    uint32_t packed[2] = {0, 0};
#pragma unroll
    for (int e = 0; e < 8; ++e) {
        const int c = sc > 0.f ? max(-kMax, min(kMax, __float2int_rn(__fdiv_rn(y[e], sc)))) : 0;
        if constexpr (KB == 8) packed[e / 4] |= (static_cast<uint32_t>(c) & 0xffu) << (8 * (e & 3));
        else packed[e / 4] |= static_cast<uint32_t>(c + 8) << (4 * (e & 3));
    }
    if constexpr (KB == 8) {
        *reinterpret_cast<uint32_t *>(codes + a) = packed[0];
        *reinterpret_cast<uint32_t *>(codes + b) = packed[1];
    } else {
        *reinterpret_cast<uint16_t *>(codes + a / 2) = static_cast<uint16_t>(packed[0]);
        *reinterpret_cast<uint16_t *>(codes + b / 2) = static_cast<uint16_t>(packed[1]);
    }
    if (l == 0) *scale = sc;
}

struct TokenPlace {
    int seq, n, len;
    int first;  // the sequence's first packed row
};

// The sequences that own the packed rows [token, token + kWarps), from all
// sequences' query counts: each thread sums a run of them, a block-wide scan
// gives the runs' starts, and the threads whose runs hold the rows walk them.
// seq is -1 behind the last row. Block 0 also checks every sequence (each block
// skips the rows of a bad one).
__device__ __forceinline__ void locate(const RopeParams &P, int token, TokenPlace (&place)[kWarps]) {
    __shared__ long long s_total[kWarps];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int per = (P.B + kThreads - 1) / kThreads;
    const int lo = min(P.B, static_cast<int>(threadIdx.x) * per), hi = min(P.B, lo + per);
    long long sum = 0;
    for (int b = lo; b < hi; ++b) sum += max(P.q_lens[b], 0);
    const int len0 = lo < hi ? P.seq_lens[lo] : 0;
    long long incl = sum;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const long long up = __shfl_up_sync(0xffffffffu, incl, o);
        if (lane >= o) incl += up;
    }
    if (lane == 31) s_total[warp] = incl;
    if (threadIdx.x < kWarps) place[threadIdx.x].seq = -1;
    __syncthreads();
    long long at = incl - sum;
    for (int w = 0; w < warp; ++w) at += s_total[w];
    if (blockIdx.x == 0) {
        bool bad = false;
        long long a = at;
        for (int b = lo; b < hi; ++b) {
            const int n = P.q_lens[b];
            a += max(n, 0);
            bad |= n < 0 || n > P.seq_lens[b] || n > P.max_q_len || a > P.total_q;
        }
        if (bad) flag_error(P.err, kErrBitQlen);
    }
    if (at < token + kWarps && at + sum > token) {
        for (int b = lo; b < hi && at < token + kWarps; ++b) {
            const int n = max(P.q_lens[b], 0);
            for (int k = 0; k < kWarps; ++k)
                if (token + k >= at && token + k < at + n)
                    place[k] = TokenPlace{b, n, b == lo ? len0 : P.seq_lens[b], static_cast<int>(at)};
            at += n;
        }
    }
    __syncthreads();
}

// KB: 0 for dense keys (no pages), 16 for bf16 pages, 8 or 4 for code pages.
template <int KB, bool kInterleaved>
__global__ void __launch_bounds__(kThreads, 8) rope_kernel(const RopeParams P) {
    __shared__ __align__(16) float s_cos[kWarps][kHeadDim / 2], s_sin[kWarps][kHeadDim / 2];
    // the attention kernel that follows reads q and the pages only after this
    // grid has completed
    if constexpr (KB != 0) asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int l = lane & 15, side = lane >> 4;
    const uint32_t mask = 0xffffu << (lane & 16);
    const int64_t gw = static_cast<int64_t>(blockIdx.x) * kWarps + warp;
    const int parts = 1 << P.parts_log2;
    const int token = static_cast<int>(gw >> P.parts_log2);
    const int part = static_cast<int>(gw) & (parts - 1);
    // two angles a lane
    const float freq0 = lane < P.half ? P.inv_freq[lane] : 0.f;
    const float freq1 = lane + 32 < P.half ? P.inv_freq[lane + 32] : 0.f;

    int pos, pid = 0, slot = 0;
    if constexpr (KB == 0) {
        if (token >= P.total_q) return;
        pos = P.positions[token];
    } else {
        __shared__ TokenPlace s_place[kWarps];
        const int token0 = static_cast<int>(static_cast<int64_t>(blockIdx.x) * kWarps >> P.parts_log2);
        locate(P, token0, s_place);
        if (token >= P.total_q) return;
        const TokenPlace at = s_place[token - token0];
        if (at.seq < 0 || at.n > at.len || at.n > P.max_q_len || at.first + static_cast<long long>(at.n) > P.total_q)
            return;
        pos = at.len - at.n + (token - at.first);
        const int j = pos / kPageSize;
        slot = pos % kPageSize;
        pid = j < P.max_pages ? P.block_table[static_cast<int64_t>(at.seq) * P.max_pages + j] : -1;
        if (P.positions != nullptr) pos = P.positions[token];
    }

    // where the lane's values stand in a row: the pairs' first and second values
    // (half a rotation apart, or neighbours), behind them eight in a row
    const bool rot = l < P.half / 4;
    const int off_a = kInterleaved || !rot ? 8 * l : 4 * l;
    const int off_b = kInterleaved || !rot ? off_a + 4 : P.half + 4 * l;
    // groups of row pairs: the queries', then the keys' with the values'
    const int nq = (P.Hq + 1) / 2, nk = (P.Hkv + 1) / 2;
    const int gq = (nq + kGroup - 1) / kGroup;
    constexpr int kKeys = KB == 0 ? kGroup : kGroup / 2;  // key pairs of a group
    const int groups = gq + (nk + kKeys - 1) / kKeys;
    const uint16_t *q = P.q + token * P.q_stride + side * kHeadDim;
    const uint16_t *k = P.k + token * P.k_stride + side * kHeadDim;
    const uint16_t *v = KB == 0 ? nullptr : P.v + token * P.v_stride + side * kHeadDim;
    // the head of a group's u-th row, and whether the row is there (a whole half warp)
    auto head_of = [&](int g, int u) {
        return 2 * (g < gq ? g * kGroup + u : (g - gq) * kKeys + (u & (kKeys - 1))) + side;
    };
    uint2 ra[kGroup], rb[kGroup];
    auto load = [&](int g, uint2 (&a)[kGroup], uint2 (&b)[kGroup]) {
        const int heads = g < gq ? P.Hq : P.Hkv;
#pragma unroll
        for (int u = 0; u < kGroup; ++u) {
            const int h = head_of(g, u);
            const uint16_t *src = (g < gq ? q : u < kKeys ? k : v) + (h - side) * kHeadDim;
            a[u] = b[u] = make_uint2(0, 0);
            if (g < groups && h < heads) {
                if constexpr (kInterleaved) {
                    const uint4 r = *reinterpret_cast<const uint4 *>(src + off_a);
                    a[u] = make_uint2(r.x, r.y);
                    b[u] = make_uint2(r.z, r.w);
                } else {
                    a[u] = *reinterpret_cast<const uint2 *>(src + off_a);
                    b[u] = *reinterpret_cast<const uint2 *>(src + off_b);
                }
            }
        }
    };
    load(part, ra, rb);

    // the token's angles, while the first rows are on their way
    auto angle = [&](float freq, int j) {
        const double turns = static_cast<double>(pos) * (static_cast<double>(freq) * 0.15915494309189535);
        sincospif(static_cast<float>(2.0 * (turns - rint(turns))), &s_sin[warp][j], &s_cos[warp][j]);
    };
    if (lane < P.half) angle(freq0, lane);
    if (lane + 32 < P.half) angle(freq1, lane + 32);
    __syncwarp();
    Turn T;
    auto prepare = [&](const float *weight) {
        float4 wa = make_float4(1.f, 1.f, 1.f, 1.f), wb = wa;
        if (weight != nullptr) {
            wa = __ldg(reinterpret_cast<const float4 *>(weight + off_a));
            wb = __ldg(reinterpret_cast<const float4 *>(weight + off_b));
        }
        const uint64_t A[2] = {kInterleaved ? two(wa.x, wa.z) : two(wa.x, wa.y), kInterleaved ? two(wb.x, wb.z) : two(wa.z, wa.w)};
        const uint64_t B[2] = {kInterleaved ? two(wa.y, wa.w) : two(wb.x, wb.y), kInterleaved ? two(wb.y, wb.w) : two(wb.z, wb.w)};
        float4 c = make_float4(1.f, 1.f, 1.f, 1.f), s = make_float4(0.f, 0.f, 0.f, 0.f);
        if (rot) {
            c = *reinterpret_cast<const float4 *>(&s_cos[warp][4 * l]);
            s = *reinterpret_cast<const float4 *>(&s_sin[warp][4 * l]);
        }
        const uint64_t C[2] = {two(c.x, c.y), two(c.z, c.w)}, S[2] = {two(s.x, s.y), two(s.z, s.w)};
        const uint64_t minus = two(-1.f, -1.f);
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            T.ac[i] = mul2(A[i], C[i]);
            T.as[i] = mul2(A[i], S[i]);
            T.bc[i] = mul2(B[i], C[i]);
            T.bs[i] = mul2(mul2(B[i], S[i]), minus);
        }
    };
    int prepared = -1;
    for (int g = part; g < groups; g += parts) {
        uint2 na[kGroup], nb[kGroup];
        load(g + parts, na, nb);
        const bool queries = g < gq;
        const float *weight = queries ? P.q_weight : P.k_weight;
        if (prepared != static_cast<int>(queries)) {
            prepare(weight);
            prepared = queries;
        }
        const int heads = queries ? P.Hq : P.Hkv;
#pragma unroll
        for (int u = 0; u < kGroup; ++u) {
            const int head = head_of(g, u);
            const bool value = !queries && u >= kKeys;
            uint2 oa = ra[u], ob = rb[u];
            float y[8];
            if (!value) {
                Eight x = unpack<kInterleaved>(ra[u], rb[u]);
                const float r = weight != nullptr ? norm_factor(x, P.eps, mask) : 1.f;
                if (rot) {
#pragma unroll
                    for (int i = 0; i < 2; ++i) {
                        const uint64_t A = fma2(x.A[i], T.ac[i], mul2(x.B[i], T.bs[i]));
                        x.B[i] = fma2(x.A[i], T.as[i], mul2(x.B[i], T.bc[i]));
                        x.A[i] = A;
                    }
                } else {
#pragma unroll
                    for (int i = 0; i < 2; ++i) {
                        x.A[i] = mul2(x.A[i], T.ac[i]);
                        x.B[i] = mul2(x.B[i], T.bc[i]);
                    }
                }
                const uint64_t rr = two(r, r);
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                    x.A[i] = mul2(x.A[i], rr);
                    x.B[i] = mul2(x.B[i], rr);
                }
                in_order<kInterleaved>(x, y);
                oa = make_uint2(pack_bf16x2(y[0], y[1]), pack_bf16x2(y[2], y[3]));
                ob = make_uint2(pack_bf16x2(y[4], y[5]), pack_bf16x2(y[6], y[7]));
            } else if constexpr (KB == 8 || KB == 4) {
                y[0] = bf16_lo(oa.x), y[1] = bf16_hi(oa.x), y[2] = bf16_lo(oa.y), y[3] = bf16_hi(oa.y);
                y[4] = bf16_lo(ob.x), y[5] = bf16_hi(ob.x), y[6] = bf16_lo(ob.y), y[7] = bf16_hi(ob.y);
            }
            auto store_row = [&](uint16_t *row) {
                if constexpr (kInterleaved) {
                    *reinterpret_cast<uint4 *>(row + off_a) = make_uint4(oa.x, oa.y, ob.x, ob.y);
                } else {
                    *reinterpret_cast<uint2 *>(row + off_a) = oa;
                    *reinterpret_cast<uint2 *>(row + off_b) = ob;
                }
            };
            if (head >= heads) continue;
            if (queries) {
                store_row(P.q_out + token * P.q_out_stride + head * kHeadDim);
            } else if constexpr (KB == 0) {
                store_row(P.k_out + token * P.k_out_stride + head * kHeadDim);
            } else if (pid < 0 || pid >= P.num_pages) {
                if (l == 0) flag_error(P.err, kErrBitPageOOB);
            } else {
                const int64_t prow = (static_cast<int64_t>(pid) * P.Hkv + head) * kPageSize + slot;
                if constexpr (KB == 16) {
                    store_row((value ? P.v_pages : P.k_pages) + prow * kHeadDim);
                } else {
                    constexpr int kCodeRow = kHeadDim * KB / 8;
                    store_codes<KB>(y, l, off_a, off_b, mask, (value ? P.v_codes : P.k_codes) + prow * kCodeRow,
                                    (value ? P.v_scales : P.k_scales) + prow);
                }
            }
        }
#pragma unroll
        for (int u = 0; u < kGroup; ++u) ra[u] = na[u], rb[u] = nb[u];
    }
}

template <bool kInterleaved>
auto kernel_for(int code_bits) {
    return code_bits == 0    ? rope_kernel<0, kInterleaved>
           : code_bits == 16 ? rope_kernel<16, kInterleaved>
           : code_bits == 8  ? rope_kernel<8, kInterleaved>
                             : rope_kernel<4, kInterleaved>;
}

}  // namespace

cudaError_t launch_rope(RopeParams p, int code_bits, int sms, cudaStream_t stream) {
    // Warps a token: what takes the fewest rounds of the resident warps, a
    // round lasting its groups and about two groups' time of start.
    const int slots = sms * 8 * kWarps;
    const int keys = code_bits == 0 ? kGroup : kGroup / 2;
    const int groups = ((p.Hq + 1) / 2 + kGroup - 1) / kGroup + ((p.Hkv + 1) / 2 + keys - 1) / keys;
    int64_t best = INT64_MAX;
    for (int log2 = 0; log2 <= 3; ++log2) {
        const int64_t warps = static_cast<int64_t>(p.total_q) << log2;
        const int64_t cost = (warps + slots - 1) / slots * (2 + (groups + (1 << log2) - 1) / (1 << log2));
        if (cost < best) {
            best = cost;
            p.parts_log2 = log2;
        }
    }
    const int64_t warps = static_cast<int64_t>(p.total_q) << p.parts_log2;
    auto kernel = p.interleaved ? kernel_for<true>(code_bits) : kernel_for<false>(code_bits);
    kernel<<<static_cast<unsigned>((warps + kWarps - 1) / kWarps), kThreads, 0, stream>>>(p);
    return cudaGetLastError();
}

}  // namespace sa
