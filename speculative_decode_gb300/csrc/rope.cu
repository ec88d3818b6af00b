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
// Half a warp holds a row, 16 bytes a lane; a CTA takes one token, whose
// angles its first threads compute once for all heads. Bound: bytes moved (a
// row in, a row out) for many tokens, two dependent memory round trips
// (lengths, then rows) for few.
#include <cfloat>

#include "common.cuh"

namespace sa {

namespace {

constexpr int kThreads = 256;
constexpr int kGroups = kThreads / 16;  // rows in one step of a CTA
constexpr int kUnroll = 3;              // rows in flight per lane

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
__device__ __forceinline__ void norm_row(float (&y)[8], const float *w, float eps, int l, uint32_t mask) {
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
    const float4 w0 = __ldg(reinterpret_cast<const float4 *>(w + 8 * l));
    const float4 w1 = __ldg(reinterpret_cast<const float4 *>(w + 8 * l) + 1);
    y[0] *= r * w0.x;
    y[1] *= r * w0.y;
    y[2] *= r * w0.z;
    y[3] *= r * w0.w;
    y[4] *= r * w1.x;
    y[5] *= r * w1.y;
    y[6] *= r * w1.z;
    y[7] *= r * w1.w;
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

// The sequence that owns a packed row, from all sequences' query counts: each
// thread sums a run of them, a block-wide scan gives the runs' starts, and the
// thread whose run holds the row walks it. seq is -1 behind the last row. CTA 0
// also checks every sequence (each other CTA skips the rows of a bad one).
__device__ __forceinline__ TokenPlace locate(const RopeParams &P, int token) {
    __shared__ long long s_total[kThreads / 32];
    __shared__ TokenPlace s_place;
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
    if (threadIdx.x == 0) s_place.seq = -1;
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
    if (token >= at && token < at + sum) {
        int b = lo;
        while (token >= at + max(P.q_lens[b], 0)) at += max(P.q_lens[b++], 0);
        s_place = TokenPlace{b, P.q_lens[b], b == lo ? len0 : P.seq_lens[b], static_cast<int>(at)};
    }
    __syncthreads();
    return s_place;
}

// KB: 0 for dense keys (no pages), 16 for bf16 pages, 8 or 4 for code pages.
template <int KB>
__global__ void __launch_bounds__(kThreads) rope_kernel(const RopeParams P) {
    __shared__ __align__(16) float s_cos[kHeadDim / 2], s_sin[kHeadDim / 2];
    // the attention kernel that follows reads q and the pages only after this
    // grid has completed
    if constexpr (KB != 0) asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    const int token = blockIdx.x;
    const int l = threadIdx.x & 15;
    const int group = threadIdx.x >> 4;
    const uint32_t mask = 0xffffu << (threadIdx.x & 16);
    const float freq = threadIdx.x < P.half ? P.inv_freq[threadIdx.x] : 0.f;

    int pos, pid = 0, slot = 0;
    if constexpr (KB == 0) {
        pos = P.positions[token];
    } else {
        const TokenPlace at = locate(P, token);
        if (at.seq < 0 || at.n > at.len || at.n > P.max_q_len || at.first + static_cast<long long>(at.n) > P.total_q)
            return;
        pos = at.len - at.n + (token - at.first);
        const int j = pos / kPageSize;
        slot = pos % kPageSize;
        pid = j < P.max_pages ? P.block_table[static_cast<int64_t>(at.seq) * P.max_pages + j] : -1;
        if (P.positions != nullptr) pos = P.positions[token];
    }

    const int rows = P.Hq + (KB == 0 ? P.Hkv : 2 * P.Hkv);
    bool turned = false;  // the angles are in shared memory
    float c[8], s[8];
    const int sh = P.half / 8;
    const bool rot = l < 2 * sh;
    for (int r0 = group; r0 - group < rows; r0 += kGroups * kUnroll) {
        uint4 raw[kUnroll];
#pragma unroll
        for (int u = 0; u < kUnroll; ++u) {
            const int r = r0 + u * kGroups;
            const uint16_t *src = r < P.Hq          ? P.q + token * P.q_stride + r * kHeadDim
                                  : r < P.Hq + P.Hkv ? P.k + token * P.k_stride + (r - P.Hq) * kHeadDim
                                                     : P.v + token * P.v_stride + (r - P.Hq - P.Hkv) * kHeadDim;
            raw[u] = r < rows ? *reinterpret_cast<const uint4 *>(src + 8 * l) : make_uint4(0, 0, 0, 0);
        }
        if (!turned) {  // while the first rows are on their way
            if (threadIdx.x < P.half) {
                const double turns = static_cast<double>(pos) * (static_cast<double>(freq) * 0.15915494309189535);
                const float part = static_cast<float>(2.0 * (turns - rint(turns)));
                sincospif(part, &s_sin[threadIdx.x], &s_cos[threadIdx.x]);
            }
            __syncthreads();
            turned = true;
            if (rot) {
                const int j = P.interleaved ? 4 * l : 8 * (l < sh ? l : l - sh);
#pragma unroll
                for (int e = 0; e < 8; ++e) {
                    const int je = P.interleaved ? j + e / 2 : j + e;
                    c[e] = s_cos[je];
                    const bool second = P.interleaved ? (e & 1) : l >= sh;
                    s[e] = second ? s_sin[je] : -s_sin[je];
                }
            }
        }
#pragma unroll
        for (int u = 0; u < kUnroll; ++u) {
            const int r = r0 + u * kGroups;
            if (r >= rows) continue;  // a whole half warp
            const bool is_q = r < P.Hq, is_v = r >= P.Hq + P.Hkv;
            float y[8] = {bf16_lo(raw[u].x), bf16_hi(raw[u].x), bf16_lo(raw[u].y), bf16_hi(raw[u].y),
                          bf16_lo(raw[u].z), bf16_hi(raw[u].z), bf16_lo(raw[u].w), bf16_hi(raw[u].w)};
            uint4 packed = raw[u];
            if (!is_v) {
                const float *w = is_q ? P.q_weight : P.k_weight;
                if (w != nullptr) norm_row(y, w, P.eps, l, mask);
                float p[8];
                if (P.interleaved) {
#pragma unroll
                    for (int e = 0; e < 8; ++e) p[e] = y[e ^ 1];
                } else {
                    const int other = !rot ? l : l < sh ? l + sh : l - sh;
#pragma unroll
                    for (int e = 0; e < 8; ++e) p[e] = __shfl_sync(mask, y[e], other, 16);
                }
                if (rot) {
#pragma unroll
                    for (int e = 0; e < 8; ++e) y[e] = fmaf(y[e], c[e], p[e] * s[e]);
                }
                packed = make_uint4(pack_bf16x2(y[0], y[1]), pack_bf16x2(y[2], y[3]), pack_bf16x2(y[4], y[5]),
                                    pack_bf16x2(y[6], y[7]));
            }
            if (is_q) {
                *reinterpret_cast<uint4 *>(P.q_out + token * P.q_out_stride + r * kHeadDim + 8 * l) = packed;
                continue;
            }
            if constexpr (KB == 0) {
                *reinterpret_cast<uint4 *>(P.k_out + token * P.k_out_stride + (r - P.Hq) * kHeadDim + 8 * l) = packed;
            } else {
                if (pid < 0 || pid >= P.num_pages) {
                    if (l == 0) flag_error(P.err, kErrBitPageOOB);
                    continue;
                }
                const int g = is_v ? r - P.Hq - P.Hkv : r - P.Hq;
                const int64_t prow = (static_cast<int64_t>(pid) * P.Hkv + g) * kPageSize + slot;
                if constexpr (KB == 16) {
                    uint16_t *pages = is_v ? P.v_pages : P.k_pages;
                    *reinterpret_cast<uint4 *>(pages + prow * kHeadDim + 8 * l) = packed;
                } else {
                    constexpr int kCodeRow = kHeadDim * KB / 8;
                    store_codes<KB>(y, l, mask, (is_v ? P.v_codes : P.k_codes) + prow * kCodeRow,
                                    (is_v ? P.v_scales : P.k_scales) + prow);
                }
            }
        }
    }
}

}  // namespace

cudaError_t launch_rope(const RopeParams &p, int code_bits, int num_tokens, cudaStream_t stream) {
    auto kernel = code_bits == 0    ? rope_kernel<0>
                  : code_bits == 16 ? rope_kernel<16>
                  : code_bits == 8  ? rope_kernel<8>
                                    : rope_kernel<4>;
    kernel<<<num_tokens, kThreads, 0, stream>>>(p);
    return cudaGetLastError();
}

}  // namespace sa
