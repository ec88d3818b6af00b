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
// Half a warp holds a row, 16 bytes a lane. A warp takes one token, or every
// `parts`-th pair of a token's rows where there are few tokens: its lanes
// compute the token's angles once for all its rows, and no warp waits for
// another after the token's sequence is found. Bound: bytes moved (a row in, a row
// out) for many tokens, two dependent memory round trips (lengths, then rows)
// for few.
#include <cfloat>

#include "common.cuh"

namespace sa {

namespace {

constexpr int kThreads = 128;
constexpr int kWarps = kThreads / 32;
constexpr int kFlight = 4;  // row pairs in flight per warp

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

// y = x * rsqrt(mean(x^2) + eps) * w for the half warp's row. A sum of squares
// past 32 bits is formed again of scaled values (a power of two), so rows of
// any finite values have their norm.
__device__ __forceinline__ void norm_row(float (&y)[8], const float (&w)[8], float eps, uint32_t mask) {
    float ss = 0.f;
#pragma unroll
    for (int e = 0; e < 8; ++e) ss = fmaf(y[e], y[e], ss);
    ss = half_warp_sum(ss, mask);
    float r = rsqrtf(fmaf(ss, 1.f / kHeadDim, eps));
    if (!(ss <= FLT_MAX)) {
        constexpr float kDown = 0x1p-70f;
        float s2 = 0.f;
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            y[e] *= kDown;
            s2 = fmaf(y[e], y[e], s2);
        }
        s2 = half_warp_sum(s2, mask);
        r = rsqrtf(s2 * (1.f / kHeadDim));  // eps is far below such a row's mean
    }
#pragma unroll
    for (int e = 0; e < 8; ++e) y[e] *= r * w[e];
}

// The page format of the quantising appends (see kv_append.cu), half a warp a
// row: scale = amax / Cmax and code = round-half-even(y / scale), both by IEEE
// division.
template <int KB>
__device__ __forceinline__ void store_codes(const float (&y)[8], int l, uint32_t mask, uint8_t *codes,
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
        else packed[0] |= static_cast<uint32_t>(c + 8) << (4 * e);
    }
    if constexpr (KB == 8) *reinterpret_cast<uint2 *>(codes + 8 * l) = make_uint2(packed[0], packed[1]);
    else *reinterpret_cast<uint32_t *>(codes + 4 * l) = packed[0];
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
template <int KB>
__global__ void __launch_bounds__(kThreads) rope_kernel(const RopeParams P) {
    __shared__ __align__(16) float s_cos[kWarps][kHeadDim / 2], s_sin[kWarps][kHeadDim / 2];
    // the attention kernel that follows reads q and the pages only after this
    // grid has completed
    if constexpr (KB != 0) asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int l = lane & 15, side = lane >> 4;
    const uint32_t mask = 0xffffu << (lane & 16);
    const int64_t gw = static_cast<int64_t>(blockIdx.x) * kWarps + warp;
    const int token = static_cast<int>(gw >> P.parts_log2);
    const int part = static_cast<int>(gw) & ((1 << P.parts_log2) - 1);
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

    // pairs of rows: the queries', the keys', then the values'
    const int nq = (P.Hq + 1) / 2, nk = (P.Hkv + 1) / 2;
    const int pairs = nq + (KB == 0 ? nk : 2 * nk);
    const int parts = 1 << P.parts_log2;
    const uint16_t *q = P.q + token * P.q_stride + 8 * l;
    const uint16_t *k = P.k + token * P.k_stride + 8 * l;
    const uint16_t *v = P.v + token * P.v_stride + 8 * l;
    bool turned = false;  // the angles are there
    float c[8], s[8], w[8];
    int w_of = -1;        // whose weights w holds: 0 queries, 1 keys
    const int sh = P.half / 8;
    const bool rot = l < 2 * sh;
    const int other = !rot || P.interleaved ? l : l < sh ? l + sh : l - sh;
    for (int p0 = part; p0 < pairs; p0 += parts * kFlight) {
        uint4 raw[kFlight];
#pragma unroll
        for (int u = 0; u < kFlight; ++u) {
            const int p = p0 + u * parts;
            const int kind = p < nq ? 0 : p < nq + nk ? 1 : 2;
            const int head = 2 * (p - (kind == 0 ? 0 : kind == 1 ? nq : nq + nk)) + side;
            const uint16_t *src = (kind == 0 ? q : kind == 1 ? k : v) + head * kHeadDim;
            raw[u] = p < pairs && head < (kind == 0 ? P.Hq : P.Hkv) ? *reinterpret_cast<const uint4 *>(src)
                                                                   : make_uint4(0, 0, 0, 0);
        }
        if (!turned) {  // while the first rows are on their way
            const double to_turns = 0.15915494309189535;
            auto turn = [&](float freq, int j) {
                const double turns = static_cast<double>(pos) * (static_cast<double>(freq) * to_turns);
                sincospif(static_cast<float>(2.0 * (turns - rint(turns))), &s_sin[warp][j], &s_cos[warp][j]);
            };
            if (lane < P.half) turn(freq0, lane);
            if (lane + 32 < P.half) turn(freq1, lane + 32);
            __syncwarp();
            turned = true;
            if (rot) {
                const int j = P.interleaved ? 4 * l : 8 * (l < sh ? l : l - sh);
#pragma unroll
                for (int e = 0; e < 8; ++e) {
                    const int je = P.interleaved ? j + e / 2 : j + e;
                    const bool second = P.interleaved ? (e & 1) : l >= sh;
                    c[e] = s_cos[warp][je];
                    s[e] = second ? s_sin[warp][je] : -s_sin[warp][je];
                }
            }
        }
#pragma unroll
        for (int u = 0; u < kFlight; ++u) {
            const int p = p0 + u * parts;
            if (p >= pairs) break;
            const int kind = p < nq ? 0 : p < nq + nk ? 1 : 2;
            const int head = 2 * (p - (kind == 0 ? 0 : kind == 1 ? nq : nq + nk)) + side;
            const bool here = head < (kind == 0 ? P.Hq : P.Hkv);  // a whole half warp
            float y[8] = {bf16_lo(raw[u].x), bf16_hi(raw[u].x), bf16_lo(raw[u].y), bf16_hi(raw[u].y),
                          bf16_lo(raw[u].z), bf16_hi(raw[u].z), bf16_lo(raw[u].w), bf16_hi(raw[u].w)};
            uint4 packed = raw[u];
            if (kind != 2) {
                const float *weight = kind == 0 ? P.q_weight : P.k_weight;
                if (weight != nullptr) {
                    if (w_of != kind) {
                        const float4 a = __ldg(reinterpret_cast<const float4 *>(weight + 8 * l));
                        const float4 b = __ldg(reinterpret_cast<const float4 *>(weight + 8 * l) + 1);
                        w[0] = a.x, w[1] = a.y, w[2] = a.z, w[3] = a.w;
                        w[4] = b.x, w[5] = b.y, w[6] = b.z, w[7] = b.w;
                        w_of = kind;
                    }
                    norm_row(y, w, P.eps, mask);
                }
                float o[8];
                if (P.interleaved) {
#pragma unroll
                    for (int e = 0; e < 8; ++e) o[e] = y[e ^ 1];
                } else {
#pragma unroll
                    for (int e = 0; e < 8; ++e) o[e] = __shfl_sync(mask, y[e], other, 16);
                }
                if (rot) {
#pragma unroll
                    for (int e = 0; e < 8; ++e) y[e] = fmaf(y[e], c[e], o[e] * s[e]);
                }
                packed = make_uint4(pack_bf16x2(y[0], y[1]), pack_bf16x2(y[2], y[3]), pack_bf16x2(y[4], y[5]),
                                    pack_bf16x2(y[6], y[7]));
            }
            if (!here) continue;
            if (kind == 0) {
                *reinterpret_cast<uint4 *>(P.q_out + token * P.q_out_stride + head * kHeadDim + 8 * l) = packed;
                continue;
            }
            if constexpr (KB == 0) {
                *reinterpret_cast<uint4 *>(P.k_out + token * P.k_out_stride + head * kHeadDim + 8 * l) = packed;
            } else {
                if (pid < 0 || pid >= P.num_pages) {
                    if (l == 0) flag_error(P.err, kErrBitPageOOB);
                    continue;
                }
                const int64_t prow = (static_cast<int64_t>(pid) * P.Hkv + head) * kPageSize + slot;
                if constexpr (KB == 16) {
                    uint16_t *pages = kind == 2 ? P.v_pages : P.k_pages;
                    *reinterpret_cast<uint4 *>(pages + prow * kHeadDim + 8 * l) = packed;
                } else {
                    constexpr int kCodeRow = kHeadDim * KB / 8;
                    store_codes<KB>(y, l, mask, (kind == 2 ? P.v_codes : P.k_codes) + prow * kCodeRow,
                                    (kind == 2 ? P.v_scales : P.k_scales) + prow);
                }
            }
        }
    }
}

}  // namespace

cudaError_t launch_rope(RopeParams p, int code_bits, int sms, cudaStream_t stream) {
    // a warp a token, and up to eight where that leaves SMs with few warps
    int log2 = 0;
    while (log2 < 3 && (static_cast<int64_t>(p.total_q) << log2) < 12ll * sms) ++log2;
    p.parts_log2 = log2;
    const int64_t warps = static_cast<int64_t>(p.total_q) << log2;
    auto kernel = code_bits == 0    ? rope_kernel<0>
                  : code_bits == 16 ? rope_kernel<16>
                  : code_bits == 8  ? rope_kernel<8>
                                    : rope_kernel<4>;
    kernel<<<static_cast<unsigned>((warps + kWarps - 1) / kWarps), kThreads, 0, stream>>>(p);
    return cudaGetLastError();
}

}  // namespace sa
