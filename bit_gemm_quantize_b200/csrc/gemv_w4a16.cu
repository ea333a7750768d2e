// Products of a few unquantized tokens (fp32, fp16 or bf16) with the packed
// 4-bit weights, for one layer or for every expert over its routed rows:
//   y[m,n] = sum_g s[g,n] * P_g[m,n],   P_g[m,n] = sum_{k in g} x[m,k] q[k,n]
// with fp32 group scales s = s_g, or s = S / alpha from the integer ones.
//
// Bound by HBM if the arithmetic behind the weight stream stays small: at the
// copy rate an SM gets 2 KB of weights (4096 codes) every 90 cycles, 350 issue
// slots.  Turning the codes into 16-bit floats for the floating-point MMA takes
// 11 instructions per 8 codes, 7 of them on the half-rate integer pipe: that
// alone is the whole time (measured 18.8 us against 7.4 us of HBM at one token,
// K = 4096, N = 22016).  The codes as int8 (16 q, three instructions per 8
// codes, as the W4A8 kernels unpack them) feed mma.sync m16n8k32 s8 instead, at
// the same rate per instruction and twice the K; so the tokens become integers.
//
// Tokens as integers: each block of 128 values of a token is written as
//   x[k] = v[k] * 2^e + r[k],  v = rne(x / 2^e),  2^e = 2^-29 of the power of two
// below the block's largest magnitude: 30 bits and a sign, |r| <= 2^-30 of that
// largest magnitude.  fp16 and bf16 values that are at least 2^-19 or 2^-22 of
// the block's largest, and fp32 values at least 2^-6 of it, are kept exactly; an
// fp32 sum of the products would round at 2^-24 of the largest one.  (Blocks whose
// largest value is below 2^-108, or 2^-115 alpha, keep fewer bits.)  The cut is relative to the largest
// value, also where a code of 0 keeps that one out of the product: a token with a
// block of a few large values over much smaller ones is multiplied again in fp32
// (few_large, plain_runs), so that elsewhere a cut is within 2^-20 of the largest of
// the eight values around it, or of the average of the block.  v is split into
// four signed 8-bit digits, each a column of the MMA, so all sums over a block
// are exact in int32.  Pairs of digits are joined exactly (c1 * 256 + c0 < 2^30),
// converted to fp32 and scaled:
//   acc += s[g,n] * (F[m, block] * float(pair)),   F a power of two
// One or two tokens take one MMA column tile (8 columns), a lane holding one pair
// of a token's digits; more take pairs of tiles, digits 0 and 1 of four tokens in
// one, 2 and 3 in the other, so that a lane holds all digits of its token.
// A block with a NaN has F = NaN.  A token with a block of infinities is multiplied
// again in fp32, too, so that infinities, the zeros that they meet among the codes, and
// each other give what the formula gives.
//
// Layout.  A cluster of 1 to 8 CTAs of 16 warps (one CTA per SM) owns a range of
// columns, a multiple of 8 wide, so that the clusters' shares differ by 8
// columns at most.  Its CTAs split K; each walks the range in tiles of 32
// columns and splits its part of K over its warps in 128-wide blocks (block kb
// belongs to warp kb mod ks; with fewer blocks than warps the other warps take
// tiles of their own).  In a block, lane (g, t) = (lane / 4, lane % 4)
// loads the 32 codes k = 32 t .. 32 t + 31 of columns g, g + 8, g + 16 and
// g + 24 as 16-byte loads: a warp's load reads 64 bytes of each of 8 columns,
// the CTA's warps neighbouring pieces.  The MMA's order of K is free as long as
// both operands agree: a word's low nibbles (k 0..3) and high nibbles (k 4..7)
// are its two K-registers as they come, and the tokens' digits are staged once
// in shared memory as the 16 bytes each lane needs (conflict-free).  Every
// cluster makes the digits of its tokens, each CTA those of its part of K: the
// more tokens and K, the more CTAs share that work (made by every CTA for all
// of K, the digits of 8 tokens at K = 4096 take longer than the weights).  The
// weights and scales of the next blocks are in flight as asynchronous copies
// into a ring of each warp's own (a lane reads back the 16 bytes that it copied
// itself); kept in registers instead they crowd out the sums, and bulk copies,
// one per column and stage by a producer warp, ran at half the rate (24 us
// against 12 at one token, K = 4096, N = 22016).
//
// The warps' sums of several tiles meet in shared memory and are added in warp
// order, the CTAs' sums of a run's columns in distributed shared memory in CTA
// order.  Tokens that do not fit the shared memory for all of a CTA's K are
// staged in panels, with the columns' sums kept in shared memory between them.
//
// Measured (in a row, weights from HBM): K = 4096, N = 22016: one token 12.2 us
// (7.4 us of HBM at the copy rate; the first weights are requested only after the
// previous kernel has ended), 3 tokens 14.9, 8 tokens 20.9 to 21.9, 16 tokens (two
// passes) 36; K = 11008, N = 4096, 8 tokens 18.6; two of eight experts of K = 4096,
// N = 14336 for one token 16.4 (9.4 of HBM), all eight for 16 tokens 50 to 59 as the
// routing has it (39).  Two CTAs of 8 warps on an SM were slower (13.7 us at one token).
#include <cooperative_groups.h>
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include <cstdint>
#include <mutex>
#include <type_traits>

#include "kernels.h"
#include "moe.h"
#include "sm100_ptx.cuh"

namespace w4a8 {
namespace w4a16 {
namespace {

namespace cg = cooperative_groups;

constexpr int kWarps = 16;
constexpr int kThreads = kWarps * 32;
constexpr int kMaxCluster = 8;
constexpr int kTileCols = 32;                     // columns of a tile: two of the MMA's 16
constexpr int kStage = 2048 + 128;                // a block's weights and scales in a warp's ring
constexpr int kDepth = 3;                         // blocks in flight per warp
constexpr int rows_of(int nt) { return 2 * nt; }  // tokens of a pass with nt MMA column tiles
constexpr int kMaxRows = rows_of(4);
constexpr int kTokenBytes = 520;       // of a token's block of 128: four digits a value, two factors
constexpr int kRedStride = 40;         // floats between two tokens' 32 sums: conflict-free for the MMA's lanes
constexpr int kMaxTiles = 8;           // tiles whose sums meet at a time, at most
constexpr int kKeepBytes = 24 * 1024;  // columns' sums kept between panels of K or for the cluster's other CTAs
constexpr int kMaxExperts = 256;
constexpr int kEarlyRows = 256;        // routed rows looked up while the offsets are
constexpr int kSmemCap = 218 * 1024;   // dynamic; the static part takes up to 8 KB

// shared memory besides the tokens: the warps' rings, and their sums of a tile
// for passes of up to `rows` tokens
constexpr int kRingBytes = kWarps * kDepth * kStage;
__host__ __device__ constexpr int red_bytes(int rows) { return kWarps * rows * kRedStride * 4; }

__device__ __forceinline__ void copy16(uint32_t dst, const void* src) {
    asm volatile("cp.async.cg.shared.global.L2::128B [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
}
__device__ __forceinline__ void copy4(uint32_t dst, const void* src) {
    asm volatile("cp.async.ca.shared.global [%0], [%1], 4;" ::"r"(dst), "l"(src) : "memory");
}
__device__ __forceinline__ void copy_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
// until at most N of this thread's groups are in flight
template <int N>
__device__ __forceinline__ void copy_wait() {
    asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

// d = a * b + c on int8 operands: 16 columns x 32 codes, 32 x 8 digits
__device__ __forceinline__ void mma_s8(int (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1, int c0, int c1,
                                       int c2, int c3) {
    asm("mma.sync.aligned.m16n8k32.row.col.s32.s8.s8.s32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
        "{%10, %11, %12, %13};"
        : "=r"(d[0]), "=r"(d[1]), "=r"(d[2]), "=r"(d[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1), "r"(c0), "r"(c1), "r"(c2), "r"(c3));
}

// 8 consecutive values of a token as fp32.
__device__ __forceinline__ void load_tokens(const void* x, int type, int64_t at, float (&v)[8]) {
    if (type == kElemF32) {
        const float4* s = reinterpret_cast<const float4*>(static_cast<const float*>(x) + at);
        const float4 a = s[0], b = s[1];
        v[0] = a.x, v[1] = a.y, v[2] = a.z, v[3] = a.w;
        v[4] = b.x, v[5] = b.y, v[6] = b.z, v[7] = b.w;
    } else {
        const uint4 u = *reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(x) + at);
        const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            if (type == kElemBf16) {
                v[2 * j] = __uint_as_float(w[j] << 16);
                v[2 * j + 1] = __uint_as_float(w[j] & 0xFFFF0000u);
            } else {
                const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&w[j]));
                v[2 * j] = f.x;
                v[2 * j + 1] = f.y;
            }
        }
    }
}

// Whether a block of a token (laid out as for block_digits, E the exponent field of
// its largest magnitude, 2^(E - 127) = P) has values that digits would cut and is held
// up by so few large ones that the cut may count: with every magnitude taken at most
// as c = 2^-8 P, its nonzero values average less than c / 4.  `small`: the lanes without
// a large value; a block without such lanes has no need to be looked at.
__device__ __forceinline__ bool few_large(const float (&v)[8], int type, int E, unsigned small) {
    // magnitudes from 2^-6 P (fp32), 2^-19 P (fp16) and 2^-22 P (bf16) on keep all their bits
    const uint32_t keep = uint32_t(max(E - (type == kElemF32 ? 6 : type == kElemF16 ? 19 : 22), 1)) << 23;
    const float inv_c = __uint_as_float(uint32_t(262 - E) << 23);
    bool cut = false;
    float sum = 0.0f;  // of magnitudes, in c / 4, less the number of values that are not 0
#pragma unroll
    for (int j = 0; j < 8; ++j) {
        const float a = fabsf(v[j]);
        cut |= a != 0.0f && __float_as_uint(a) < keep;
        sum += 4.0f * __saturatef(a * inv_c) - (a != 0.0f ? 1.0f : 0.0f);
    }
#pragma unroll
    for (int o = 1; o < 32; o <<= 1)
        if (o != 4) sum += __shfl_xor_sync(0xffffffffu, sum, o);
    const unsigned lanes = (threadIdx.x & 4) ? 0xF0F0F0F0u : 0x0F0F0F0Fu;  // the block's
    return (__ballot_sync(0xffffffffu, cut) & lanes) != 0u && (small & lanes) != 0u && sum < 0.0f;
}

// A block of 128 values of one token, 8 per lane of 16 lanes (those of the warp
// that agree in bit 2), as digits: dig[d][h] holds digit d of values 4 h ..
// 4 h + 3.  Returns the factors of the low and the high pair of digits, which
// include 1/16 for the 16 q of the weights and 2^-8, so that a value next to the
// largest fp32 one does not overflow where its high pair rounds up (the output
// step multiplies by 2^8; with integer scales it is a part of 2^8 / alpha, and the
// caller multiplies the factors by the other).  Sets `plain` where the block is not for digits.
__device__ __forceinline__ float2 block_digits(const float (&v)[8], int type, uint32_t (&dig)[4][2],
                                               bool& plain) {
    uint32_t top = 0u;
#pragma unroll
    for (int j = 0; j < 8; ++j) top = max(top, __float_as_uint(v[j]) & 0x7FFFFFFFu);
    const uint32_t own = top;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1)
        if (o != 4) top = max(top, __shfl_xor_sync(0xffffffffu, top, o));
    const int E = max(int(top >> 23), 19);  // below, the factor would leave the fp32 range
    uint32_t y[8];
    float2 F;
    if (E < 255) {
        const int k = 156 - E, k1 = k / 2, k2 = k - k1;  // |v| 2^k < 2^30
        const float f1 = __uint_as_float(uint32_t(127 + k1) << 23), f2 = __uint_as_float(uint32_t(127 + k2) << 23);
#pragma unroll
        for (int j = 0; j < 8; ++j) y[j] = uint32_t(__float2int_rn(v[j] * f1 * f2));
        // 2^(E - 168): a subnormal power of two below E = 42
        F.x = E >= 42 ? __uint_as_float(uint32_t(E - 41) << 23) : __uint_as_float(1u << (E - 19));
        F.y = F.x * 65536.0f;
    } else {
#pragma unroll
        for (int j = 0; j < 8; ++j) y[j] = 0u;
        F.x = F.y = __uint_as_float(0x7FC00000u);
        if (top == 0x7F800000u) plain = true;
    }
    // signed digits: with 0x80 added to the three lower bytes (carries included)
    // and taken off again, each byte is its digit
#pragma unroll
    for (int j = 0; j < 8; ++j) y[j] = (y[j] + 0x00808080u) ^ 0x00808080u;
#pragma unroll
    for (int h = 0; h < 2; ++h) {
        const uint32_t* q = y + 4 * h;
        const uint32_t a = __byte_perm(q[0], q[1], 0x5140), b = __byte_perm(q[2], q[3], 0x5140);
        const uint32_t c = __byte_perm(q[0], q[1], 0x7362), d = __byte_perm(q[2], q[3], 0x7362);
        dig[0][h] = __byte_perm(a, b, 0x5410);
        dig[1][h] = __byte_perm(a, b, 0x7632);
        dig[2][h] = __byte_perm(c, d, 0x5410);
        dig[3][h] = __byte_perm(c, d, 0x7632);
    }
    // no need to look closer while every lane's eight values have a large one (a block's
    // answer is its own: the warp's other block must not change it).  Asked here, behind
    // the digits, it costs less: 8 tokens 18.6 us against 19.0
    const unsigned small = __ballot_sync(0xffffffffu, own < uint32_t(E - 10) << 23);
    if (small) plain |= few_large(v, type, E, small);
    return F;
}

// The tokens of one run, and where their outputs go (-1: outside, counted as
// zeros or not written).
struct Rows {
    int32_t src[kMaxRows];
    int32_t dst[kMaxRows];
    // whether this CTA, and any of the cluster, has met a block that is not for digits
    int plain, plain_all;
};

// A run: one expert's weights, up to rows_of(NT) tokens, a range of columns.
struct Run {
    const uint8_t* w;
    const void* scales;
    int32_t col0, col1;
    int m_rows;
};

// The digits and factors of a run's tokens for the blocks kb0 .. kb1 - 1: two
// (token, block) pairs per warp step, 16 lanes each; lane (xt, xw) of a pair has
// the 8 values that word xw of the weights of lanes t = xt meets.
__device__ __noinline__ void stage_tokens(const void* x, int type, int64_t ldx, Rows& rows, int m_rows, int kb0,
                                          int kb1, float scale, uint4* xs, float2* fs) {
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int xt = lane & 3, xh = (lane >> 2) & 1, xw = lane >> 3;
    const uint32_t pairs = uint32_t(m_rows * (kb1 - kb0));
    for (uint32_t q0 = warp * 2; q0 < pairs; q0 += 2 * kWarps) {
        const uint32_t q = q0 + xh;
        const uint32_t kb = q / uint32_t(m_rows), m = q - kb * m_rows;
        const int32_t row = q < pairs ? rows.src[m] : -1;
        float v[8] = {0.0f, 0.0f, 0.0f, 0.0f, 0.0f, 0.0f, 0.0f, 0.0f};
        if (row >= 0) load_tokens(x, type, int64_t(row) * ldx + int64_t(kb0 + kb) * 128 + xt * 32 + xw * 8, v);
        uint32_t dig[4][2];
        bool plain = false;
        const float2 F = block_digits(v, type, dig, plain);
        if (plain) rows.plain = 1;
        if (q < pairs) {
            uint2* dst = reinterpret_cast<uint2*>(xs + ((kb * 2 + (xw >> 1)) * m_rows + m) * 16 + xt) + (xw & 1);
#pragma unroll
            for (int d = 0; d < 4; ++d) dst[d * 8] = make_uint2(dig[d][0], dig[d][1]);
            if (xt == 0 && xw == 0) fs[q] = make_float2(F.x * scale, F.y * scale);
        }
    }
}

// 1 or 4 consecutive columns' sums (4: on 16-byte boundaries).
template <int N>
struct Cols {
    float v[N];
    __device__ __forceinline__ void add(const float* a) {
        if constexpr (N == 4) {
            const float4 f = *reinterpret_cast<const float4*>(a);
            v[0] += f.x, v[1] += f.y, v[2] += f.z, v[3] += f.w;
        } else {
            v[0] += *a;
        }
    }
    __device__ __forceinline__ void put(float* a) const {
        if constexpr (N == 4)
            *reinterpret_cast<float4*>(a) = make_float4(v[0], v[1], v[2], v[3]);
        else
            *a = v[0];
    }
};

// Columns from n of output row dst (-1: none).
template <int N>
__device__ __forceinline__ void store_out(const Params& p, int32_t dst, int32_t n, Cols<N> c) {
    if (dst < 0) return;
#pragma unroll
    for (int i = 0; i < N; ++i) c.v[i] *= p.out_scale;
    const int64_t at = int64_t(dst) * p.N + n;
    if (p.y_type == kElemF32) {
        c.put(static_cast<float*>(p.y) + at);
    } else if constexpr (N == 1) {
        if (p.y_type == kElemF16)
            static_cast<__half*>(p.y)[at] = __float2half_rn(c.v[0]);
        else
            static_cast<__nv_bfloat16*>(p.y)[at] = __float2bfloat16_rn(c.v[0]);
    } else if (p.y_type == kElemF16) {
        const __half2 a = __floats2half2_rn(c.v[0], c.v[1]), b = __floats2half2_rn(c.v[2], c.v[3]);
        *reinterpret_cast<uint2*>(static_cast<__half*>(p.y) + at) =
            make_uint2(*reinterpret_cast<const uint32_t*>(&a), *reinterpret_cast<const uint32_t*>(&b));
    } else {
        const __nv_bfloat162 a = __floats2bfloat162_rn(c.v[0], c.v[1]), b = __floats2bfloat162_rn(c.v[2], c.v[3]);
        *reinterpret_cast<uint2*>(static_cast<__nv_bfloat16*>(p.y) + at) =
            make_uint2(*reinterpret_cast<const uint32_t*>(&a), *reinterpret_cast<const uint32_t*>(&b));
    }
}

// The tokens (bits, in *found) of a run that have a block that is not for digits.
__device__ __forceinline__ void find_plain(const void* x, int type, int64_t ldx, const int32_t* src, int m_rows,
                                           int nkb, uint32_t* found) {
    const int lane = threadIdx.x & 31, xh = (lane >> 2) & 1, at = (lane & 3) * 32 + (lane >> 3) * 8;
    for (int q0 = int(threadIdx.x >> 5) * 2; q0 < m_rows * nkb; q0 += 2 * kWarps) {
        const int q = q0 + xh, m = q / nkb, kb = q - m * nkb;
        float v[8] = {0.0f, 0.0f, 0.0f, 0.0f, 0.0f, 0.0f, 0.0f, 0.0f};
        if (m < m_rows && src[m] >= 0) load_tokens(x, type, src[m] * ldx + kb * 128 + at, v);
        uint32_t dig[4][2];
        bool plain = false;
        block_digits(v, type, dig, plain);
        if (plain) atomicOr(found, 1u << m);
    }
}

// The outputs of some tokens (bits) of a run, in fp32 altogether: a warp takes four
// columns, a lane eight codes of each in a chain of products, scaled and added to the
// lane's sums; the lanes' sums are added last.  The cluster's CTAs share the columns.
// A token costs about 30 us at K = 4096, N = 22016 (bound by latency); where there is
// none, the search for it 0.2 to 0.3 us of 12 to 19.
template <bool INT>
__device__ __forceinline__ void plain_tokens(const Params& p, const Run& run, const Rows& rows, uint32_t tokens) {
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int C = 1 << p.cluster_log, rank = int(blockIdx.x) & (C - 1);
    const float scale = 0x1p-8f * p.x_scale;  // as in the factors
    for (; tokens; tokens &= tokens - 1) {
        const int m = __ffs(int(tokens)) - 1;
        const int64_t xrow = rows.src[m] * p.ldx;
        for (int32_t n = run.col0 + (rank * kWarps + warp) * 4; n < run.col1; n += C * kWarps * 4) {
            float acc[4] = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll 4
            for (int32_t k0 = lane * 8; k0 < p.K; k0 += 256) {
                float v[8];
                load_tokens(p.x, p.x_type, xrow + k0, v);
#pragma unroll
                for (int j = 0; j < 8; ++j) v[j] *= scale;
                const int kb = k0 >> 7;
                const int64_t at = int64_t(p.group_magic ? int(__umulhi(uint32_t(kb), p.group_magic)) : kb) * p.N + n;
#pragma unroll
                for (int c = 0; c < 4; ++c) {
                    const uint32_t word =
                        *reinterpret_cast<const uint32_t*>(run.w + int64_t(n + c) * (p.K >> 1) + (k0 >> 1)) ^ 0x88888888u;
                    float sum = 0.0f;
#pragma unroll
                    for (int j = 0; j < 8; ++j) {  // the low nibbles, then the high ones: q + 8, behind 2^23
                        const uint32_t code = word >> (j < 4 ? 8 * j : 8 * j - 28);
                        sum = __fmaf_rn(v[j], __uint_as_float((code & 15u) | 0x4B000000u) - 8388616.0f, sum);
                    }
                    acc[c] = __fmaf_rn(INT ? float(static_cast<const int16_t*>(run.scales)[at + c])
                                           : static_cast<const float*>(run.scales)[at + c],
                                       sum, acc[c]);
                }
            }
            Cols<4> out;
#pragma unroll
            for (int c = 0; c < 4; ++c) {
#pragma unroll
                for (int o = 16; o > 0; o >>= 1) acc[c] += __shfl_xor_sync(0xffffffffu, acc[c], o);
                out.v[c] = acc[c];
            }
            if (lane == 0) store_out(p, rows.dst[m], n, out);
        }
    }
}

// One run, with the tokens' digits in NT MMA column tiles (1 for one or two
// tokens, 2 for four, 4 for eight).
template <int NT, bool INT>
__device__ __forceinline__ void run_columns(const Params& p, const Run& run, Rows& rows, uint8_t* smem) {
    constexpr int kPair = NT == 1 ? 1 : 2;  // tiles worked on together
    constexpr int kPasses = NT / kPair;
    // columns a thread adds up at a time: with few tokens there are too few outputs to give it four
    constexpr int kColsLog = NT < 4 ? 0 : 2, kCols = 1 << kColsLog;
    // the same in every lane, and known to the compiler to be so
    const int warp = __shfl_sync(0xffffffffu, int(threadIdx.x >> 5), 0), lane = threadIdx.x & 31;
    const int g = lane >> 2, t = lane & 3;
    const int ks_log = p.ks_log, ks = 1 << ks_log, wk = warp & (ks - 1), wr = warp >> ks_log;
    const int m_rows = run.m_rows;
    // this CTA's blocks of K
    const int C = 1 << p.cluster_log, rank = int(blockIdx.x) & (C - 1), nkb = p.K >> 7;
    const int kbA = nkb * rank >> p.cluster_log, kbB = nkb * (rank + 1) >> p.cluster_log;
    const int step_log = 9 - ks_log, step_cols = 1 << step_log;  // columns of the CTA's tiles side by side
    const int64_t tile_step = int64_t(step_cols) * (p.K >> 1);  // bytes from one of this warp's tiles to its next
    // this lane's four 16-byte pieces of a block: columns g + 8 i of the tile
    uint32_t off[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) off[i] = uint32_t(g + 8 * i) * uint32_t(p.K >> 1) + uint32_t(t) * 16u;
    const uint8_t* slane = static_cast<const uint8_t*>(run.scales) + lane * 4;  // this lane's piece of a row of scales

    uint8_t* ring = smem + warp * kDepth * kStage;
    const uint32_t ring_at = smem_u32(ring);
    float* red = reinterpret_cast<float*>(smem + kRingBytes);
    const int red_warp = m_rows * kRedStride, red_tile = kWarps * red_warp;
    float* keep = red + p.red_tiles * (red_bytes(p.max_rows) / 4);  // [token][column of the batch]
    uint8_t* xbase = reinterpret_cast<uint8_t*>(keep) + (p.keeps ? kKeepBytes : 0);
    uint4* xs = reinterpret_cast<uint4*>(xbase);  // the tokens' digits, then their factors

    const int cols = 4 * m_rows;  // operand columns staged
    int panels = 1, panel_kb = (nkb + C - 1) >> p.cluster_log;  // the same for all CTAs of the cluster
    if (p.x_panels) {  // the most rows do not fit for all of K
        const int cap_kb = p.x_cap / (m_rows * kTokenBytes);
        panels = (panel_kb + cap_kb - 1) / cap_kb;
        panel_kb = (panel_kb + panels - 1) / panels;
    }
    const bool direct = panels == 1 && C == 1;  // sums go straight to y
    const int32_t batch = direct ? run.col1 - run.col0 : kKeepBytes / (4 * m_rows) >> step_log << step_log;
    float2* fs = reinterpret_cast<float2*>(xbase + panel_kb * cols * 128);  // [block][token]
    const float* fl = reinterpret_cast<const float*>(fs) + (kPair == 1 ? t & 1 : 0);  // this lane's digits

    // This lane's place in a block's digits, and its tokens' factors.  Operand
    // columns past the last token repeat it: a column's sums depend on that
    // column alone, and these are not used.
    int xlane[NT], flane[kPasses];
#pragma unroll
    for (int i = 0; i < NT; ++i) {
        const int token = kPair == 1 ? g >> 2 : 4 * (i / 2) + (g >> 1);
        const int digit = kPair == 1 ? g & 3 : (g & 1) + 2 * (i & 1);
        xlane[i] = (min(token, m_rows - 1) * 4 + digit) * 4 + t;
    }
    // this lane's token in pass i, for the products
    const auto token_of = [&](int i) { return kPair == 1 ? t >> 1 : 4 * i + t; };
#pragma unroll
    for (int i = 0; i < kPasses; ++i) flane[i] = 2 * min(token_of(i), m_rows - 1);

    for (int32_t b0 = run.col0; b0 < run.col1; b0 += batch) {
        const int32_t b1 = min(b0 + batch, run.col1);
        for (int pn = 0; pn < panels; ++pn) {
            const int kb0 = min(kbA + pn * panel_kb, kbB), kb1 = min(kb0 + panel_kb, kbB);
            const int nj = max(1, (kb1 - kb0 - wk + ks - 1) >> ks_log);  // this warp's blocks per tile (>= 1 step)

            // the tile, the block and the ring slot that load() takes next, and where they lie
            int32_t ln = b0 + wr * kTileCols;
            int lkb = kb0 + wk, lj = 0;
            uint32_t lslot = 0;
            const uint8_t* lw = run.w + (int64_t(ln) * (p.K >> 1) + lkb * 64);
            auto load = [&]() {
                if (ln < b1 && lkb < kb1) {
                    const uint32_t dst = ring_at + lslot + lane * 16;
                    const int32_t at = (p.group_magic ? int(__umulhi(uint32_t(lkb), p.group_magic)) : lkb) * p.N + ln;
                    const uint32_t sdst = ring_at + lslot + 2048 + lane * 4;
                    if (ln + kTileCols <= b1) {
#pragma unroll
                        for (int i = 0; i < 4; ++i) copy16(dst + i * 512, lw + off[i]);
                        if constexpr (INT) {
                            if (lane < 16) copy4(sdst, slane + int64_t(at) * 2);
                        } else {
                            copy4(sdst, slane + int64_t(at) * 4);
                        }
                    } else {
                        // the range's last tile: eight columns are all inside or all outside.  Outside,
                        // the slot keeps what it held, and the sums made of it are not used
#pragma unroll
                        for (int i = 0; i < 4; ++i)
                            if (ln + 8 * i < b1) copy16(dst + i * 512, lw + off[i]);
                        if (ln + (INT ? 2 * lane : lane) < b1 && (!INT || lane < 16))
                            copy4(sdst, slane + int64_t(at) * (INT ? 2 : 4));
                    }
                }
                copy_commit();
                lslot = lslot + kStage == kDepth * kStage ? 0 : lslot + kStage;
                lkb += ks;
                lw += ks * 64;
                if (++lj == nj) {
                    lj = 0;
                    lkb = kb0 + wk;
                    ln += step_cols;
                    lw += tile_step - int64_t(nj * ks) * 64;
                }
            };
#pragma unroll
            for (int u = 0; u < kDepth; ++u) load();

            if (panels > 1 || b0 == run.col0) {
                __syncthreads();  // the rows are set; the last panel's tokens have been used
                stage_tokens(p.x, p.x_type, p.ldx, rows, m_rows, kb0, kb1, p.x_scale, xs, fs);
            }
            __syncthreads();

            float acc[2][kPasses][2];  // [16-column half][pass][column g, g + 8]
#pragma unroll
            for (int r = 0; r < 2; ++r)
#pragma unroll
                for (int i = 0; i < kPasses; ++i) acc[r][i][0] = acc[r][i][1] = 0.0f;
            uint32_t cslot = 0;
            int tile = 0;  // of those whose sums wait in shared memory
            for (int32_t cn = b0; cn < b1; cn += step_cols) {  // the CTA's tiles side by side
                int ckb = wk;                                  // the block within the panel
                for (int j = 0; j < nj; ++j, ckb += ks) {
                    copy_wait<kDepth - 1>();
                    __syncwarp();  // every lane's copies of the block are there
                    if (ckb < kb1 - kb0) {
                        const uint8_t* slot = ring + cslot;
                        uint4 wreg[4];
                        std::conditional_t<INT, int, float> sreg[4];
#pragma unroll
                        for (int i = 0; i < 4; ++i) {
                            wreg[i] = *reinterpret_cast<const uint4*>(slot + i * 512 + lane * 16);
                            if constexpr (INT)
                                sreg[i] = reinterpret_cast<const int16_t*>(slot + 2048)[g + 8 * i];
                            else
                                sreg[i] = reinterpret_cast<const float*>(slot + 2048)[g + 8 * i];
                        }
                        // the codes are unpacked again for the second pair of tiles, which costs less
                        // than the registers of four tiles' sums
#pragma unroll
                        for (int pass = 0; pass < kPasses; ++pass) {
                            int c[2][kPair][4];
                            const uint4* xk = xs + ckb * 8 * cols;
#pragma unroll
                            for (int h = 0; h < 2; ++h) {
                                uint4 xv[kPair];
#pragma unroll
                                for (int i = 0; i < kPair; ++i) xv[i] = xk[h * cols * 4 + xlane[pass * kPair + i]];
#pragma unroll
                                for (int o = 0; o < 2; ++o) {  // word 2 h + o of the lane's four
#pragma unroll
                                    for (int r = 0; r < 2; ++r) {
                                        const uint4 va = wreg[2 * r], vb = wreg[2 * r + 1];
                                        const uint32_t wa = h == 0 ? (o == 0 ? va.x : va.y) : (o == 0 ? va.z : va.w);
                                        const uint32_t wb = h == 0 ? (o == 0 ? vb.x : vb.y) : (o == 0 ? vb.z : vb.w);
                                        // nibbles in the high halves of their bytes: 16 q
                                        const uint32_t a[4] = {(wa << 4) & 0xF0F0F0F0u, (wb << 4) & 0xF0F0F0F0u,
                                                               wa & 0xF0F0F0F0u, wb & 0xF0F0F0F0u};
#pragma unroll
                                        for (int i = 0; i < kPair; ++i) {
                                            int(&d)[4] = c[r][i];
                                            const uint32_t x0 = o == 0 ? xv[i].x : xv[i].z;
                                            const uint32_t x1 = o == 0 ? xv[i].y : xv[i].w;
                                            if (h == 0 && o == 0)
                                                mma_s8(d, a, x0, x1, 0, 0, 0, 0);
                                            else
                                                mma_s8(d, a, x0, x1, d[0], d[1], d[2], d[3]);
                                        }
                                    }
                                }
                            }
                            const float F = fl[ckb * 2 * m_rows + flane[pass]];
#pragma unroll
                            for (int r = 0; r < 2; ++r)
#pragma unroll
                                for (int j = 0; j < 2; ++j) {  // columns g and g + 8
                                    float v = __int2float_rn(c[r][0][2 * j + 1] * 256 + c[r][0][2 * j]);
                                    if constexpr (kPair == 2)
                                        v = __fmaf_rn(
                                            __int2float_rn(c[r][kPair - 1][2 * j + 1] * 256 + c[r][kPair - 1][2 * j]),
                                            65536.0f, v);
                                    acc[r][pass][j] = __fmaf_rn(float(sreg[2 * r + j]), __fmul_rn(F, v), acc[r][pass][j]);
                                }
                        }
                    }
                    cslot = cslot + kStage == kDepth * kStage ? 0 : cslot + kStage;
                    __syncwarp();  // every lane has used the block: its slot is free
                    load();
                }
                // the tile's sums wait for the other warps' (of one or two tokens, after the two
                // pairs of digits have met)
                float* mine = red + tile * red_tile + warp * red_warp;
#pragma unroll
                for (int i = 0; i < kPasses; ++i)
#pragma unroll
                    for (int r = 0; r < 2; ++r)
#pragma unroll
                        for (int j = 0; j < 2; ++j) {
                            float v = acc[r][i][j];
                            if constexpr (kPair == 1) v += __shfl_xor_sync(0xffffffffu, v, 1);
                            if ((kPair == 2 || (t & 1) == 0) && token_of(i) < m_rows)
                                mine[token_of(i) * kRedStride + r * 16 + j * 8 + g] = v;
                            acc[r][i][j] = 0.0f;
                        }
                if (++tile < p.red_tiles && cn + step_cols < b1) continue;
                const int32_t c0 = cn - (tile - 1) * step_cols;  // the first of the waiting tiles' columns
                __syncthreads();
                for (int o = threadIdx.x; o < tile * m_rows << (step_log - kColsLog); o += kThreads) {
                    // o: (tile, token, kCols columns of the step)
                    const int r = (o & (step_cols / kCols - 1)) * kCols, tm = o >> (step_log - kColsLog);
                    const int tl = m_rows == 1 ? tm : int(uint32_t(tm) / uint32_t(m_rows)), m = tm - tl * m_rows;
                    const int32_t n = c0 + tl * step_cols + r;
                    if (n >= b1) continue;
                    const float* part = red + tl * red_tile + (r / kTileCols << ks_log) * red_warp + m * kRedStride +
                                        (r & (kTileCols - 1));
                    Cols<kCols> sum{};
#pragma unroll 4
                    for (int i = 0; i < ks; ++i) sum.add(part + i * red_warp);
                    if (direct) {
                        store_out(p, rows.dst[m], n, sum);
                    } else {  // o's own place: until the last panel this thread alone uses it
                        float* kp = keep + m * batch + (n - b0);
                        if (pn > 0) sum.add(kp);
                        sum.put(kp);
                    }
                }
                __syncthreads();  // the sums have been read
                tile = 0;
            }
        }
        if (direct) continue;
        // the batch's sums: of all CTAs of the cluster in turn
        const int quads = (b1 - b0) / 4, n_out = quads * m_rows;
        if (C > 1) {
            cg::this_cluster().sync();  // every CTA's sums are there
            if (rows.plain && int(threadIdx.x) < C) *cg::this_cluster().map_shared_rank(&rows.plain_all, threadIdx.x) = 1;
        }
        for (int o = rank * kThreads + int(threadIdx.x); o < n_out; o += C * kThreads) {
            const int m = int(uint32_t(o) / uint32_t(quads)), n = (o - m * quads) * 4, at = m * batch + n;
            Cols<4> sum{};
            for (int i = 0; i < C; ++i) sum.add((C > 1 ? cg::this_cluster().map_shared_rank(keep, i) : keep) + at);
            store_out(p, rows.dst[m], b0 + n, sum);
        }
        if (C > 1)
            cg::this_cluster().sync();  // and have been read
        else
            __syncthreads();
    }
}

// What a CTA's threads share about the call: each expert's first routed row, the
// row chunks before its own, its weights and scales; the first routed rows, looked
// up early; the rows of the run at hand.
template <bool GROUPED>
struct Tables {
    static constexpr int kE = GROUPED ? kMaxExperts : 0, kEarly = GROUPED ? kEarlyRows : 1;
    int32_t off[kE + 1], chunk[kE + 1];
    const uint8_t* w[kE + 1];
    const void* scales[kE + 1];
    int32_t early_src[kEarly], early_dst[kEarly];
    int bad;
    Rows rows;
    // the cluster's first item, its next one and the one behind its last
    uint32_t chunks, first, it, it_end, found;
};

// The next run of the items it .. it_end - 1 (`it` moves behind it), and its rows.
template <int NT, bool GROUPED>
__device__ __forceinline__ Run next_run(const Params& p, Tables<GROUPED>& tab, uint32_t chunks, uint32_t& it,
                                        uint32_t it_end) {
    constexpr uint32_t kRows = rows_of(NT);
    const uint32_t units = uint32_t(p.N) >> 3;  // columns in eights
    Run run;
    const uint32_t chunk = !GROUPED && chunks == 1 ? 0u : it / units;
    const uint32_t unit0 = it - chunk * units;
    const uint32_t unit1 = min(units, unit0 + (it_end - it));
    it += unit1 - unit0;
    int32_t r0;
    if constexpr (GROUPED) {
        int e = 0, e_hi = p.E - 1;  // the last expert whose first chunk is <= chunk
        while (e < e_hi) {
            const int mid = (e + e_hi + 1) >> 1;
            if (tab.chunk[mid] <= int32_t(chunk)) e = mid; else e_hi = mid - 1;
        }
        r0 = tab.off[e] + int32_t((chunk - uint32_t(tab.chunk[e])) * kRows);
        run.m_rows = min(int32_t(kRows), tab.off[e + 1] - r0);
        run.w = tab.w[e];
        run.scales = tab.scales[e];
    } else {
        r0 = int32_t(chunk * kRows);
        run.m_rows = min(int32_t(kRows), int32_t(p.R) - r0);
        run.w = p.w;
        run.scales = p.scales;
    }
    run.col0 = int32_t(unit0 * 8);
    run.col1 = int32_t(unit1 * 8);

    __syncthreads();  // the last run's rows have been used
    if (int(threadIdx.x) < run.m_rows) {
        const int32_t r = r0 + int32_t(threadIdx.x);
        int32_t src = r, dst = r;
        if constexpr (GROUPED) {
            if (r < kEarlyRows) {
                src = tab.early_src[r];
                dst = tab.early_dst[r];
            } else {
                if (p.row_index) src = p.row_index[r];
                if (p.out_row) dst = p.out_row[r];
            }
        }
        if (src < 0 || src >= p.x_rows) {
            src = -1;
            atomicExch(p.status, kStatusInvalidArg);
        }
        if (dst < 0 || dst >= p.y_rows) {
            dst = -1;
            atomicExch(p.status, kStatusInvalidArg);
        }
        tab.rows.src[threadIdx.x] = src;
        tab.rows.dst[threadIdx.x] = dst;
    }
    return run;
}

// The CTA's runs once more, for the tokens that are not for digits: their outputs are
// written again, over what the digits gave.
template <int NT, bool INT, bool GROUPED>
__device__ __noinline__ void plain_runs(const Params& p, Tables<GROUPED>& tab) {
    uint32_t it = tab.first;
    while (it < tab.it_end) {
        const Run run = next_run<NT, GROUPED>(p, tab, tab.chunks, it, tab.it_end);
        if (threadIdx.x == 0) tab.found = 0u;
        __syncthreads();
        find_plain(p.x, p.x_type, p.ldx, tab.rows.src, run.m_rows, p.K >> 7, &tab.found);
        __syncthreads();
        plain_tokens<INT>(p, run, tab.rows, tab.found);
    }
}

// One kernel for each number of token tiles: together, three bodies share one
// register allocation and spill more (8 tokens 25 -> 28 us; alone, the forms for 3 and 4
// tokens spill up to 56 bytes, the one of one or two tokens per expert 4, the others
// nothing).
template <int NT, bool INT, bool GROUPED>
__global__ void __launch_bounds__(kThreads, 1) w4a16_kernel(const __grid_constant__ Params p) {
    constexpr uint32_t kRows = rows_of(NT);
    extern __shared__ __align__(128) uint8_t smem[];
    __shared__ Tables<GROUPED> tab;
    const int lane = threadIdx.x & 31;
    const uint32_t units = uint32_t(p.N) >> 3;  // columns in eights

    griddep_wait();  // tokens, routing and weights may be earlier kernels' output
    if (threadIdx.x == 0) griddep_launch_dependents();

    // ---- the row chunks of every expert
    uint32_t chunks = (uint32_t(p.R) + kRows - 1) / kRows;
    if constexpr (GROUPED) {
        if (threadIdx.x >= kThreads - kEarlyRows) {
            const int r = int(threadIdx.x) - (kThreads - kEarlyRows);
            if (r < p.R) {
                tab.early_src[r] = p.row_index ? p.row_index[r] : r;
                tab.early_dst[r] = p.out_row ? p.out_row[r] : r;
            }
        }
        if (threadIdx.x < 32) {
            int bad = 0;
            int32_t before = 0;
            for (int e0 = 0; e0 < p.E; e0 += 32) {
                const int e = e0 + lane;
                int64_t a = 0, b = 0;
                if (e < p.E) {
                    a = p.offsets[e];
                    b = p.offsets[e + 1];
                    const uint8_t* w = p.w_ptrs[e];
                    const void* sc = p.s_ptrs[e];
                    if ((e == 0 && a != 0) || a < 0 || b < a || b > p.R) bad = 1;
                    if (b > a && (!w || !sc || (reinterpret_cast<uintptr_t>(w) & 15u) != 0 ||
                                  (reinterpret_cast<uintptr_t>(sc) & 3u) != 0))
                        bad = 1;
                    tab.w[e] = w;
                    tab.scales[e] = sc;
                }
                bad = __any_sync(0xffffffffu, bad);
                if (bad) break;
                int32_t incl = int32_t((uint32_t(b - a) + kRows - 1) / kRows);
#pragma unroll
                for (int o = 1; o < 32; o <<= 1) {
                    const int32_t v = __shfl_up_sync(0xffffffffu, incl, o);
                    if (lane >= o) incl += v;
                }
                if (e < p.E) {
                    tab.off[e] = int32_t(a);
                    tab.off[e + 1] = int32_t(b);
                    tab.chunk[e + 1] = before + incl;
                }
                before += __shfl_sync(0xffffffffu, incl, 31);
            }
            if (lane == 0) {
                tab.chunk[0] = 0;
                tab.bad = bad;
                if (bad && blockIdx.x == 0) atomicExch(p.status, kStatusInvalidArg);
            }
        }
        __syncthreads();
        if (tab.bad) return;
        chunks = uint32_t(tab.chunk[p.E]);
    }

    // ---- this cluster's range of (expert, row chunk, eight columns) items, columns
    // innermost: with no more row chunks than clusters, a share of one of them
    // (a second run costs its tokens' staging once more, while the weights wait:
    // 16 us against 12 with 32 experts of one row each), else equal shares of all
    const uint32_t clusters = gridDim.x >> p.cluster_log, id = blockIdx.x >> p.cluster_log;
    uint32_t it, it_end;
    const auto share = [](uint32_t n, uint32_t parts, uint32_t i) {  // the first item of part i of n
        const uint32_t q = n / parts, more = n - q * parts;
        return i * q + min(i, more);
    };
    if (!GROUPED && chunks == 1) {
        it = share(units, clusters, id);
        it_end = share(units, clusters, id + 1);
    } else if (chunks <= clusters) {
        // cluster id belongs to chunk c: share(clusters, chunks, c) <= id < share(clusters, chunks, c + 1)
        const uint32_t q = chunks ? clusters / chunks : 1u, more = clusters - q * chunks;
        const uint32_t c = id < more * (q + 1) ? id / (q + 1) : more + (id - more * (q + 1)) / q;
        const uint32_t first = share(clusters, max(chunks, 1u), c), parts = q + (c < more ? 1u : 0u);
        it = c * units + share(units, parts, id - first);
        it_end = c * units + share(units, parts, id - first + 1);
        if (c >= chunks) it_end = it;
    } else {
        it = share(chunks * units, clusters, id);
        it_end = share(chunks * units, clusters, id + 1);
    }
    if (it >= it_end) return;
    if (threadIdx.x == 0) {
        tab.rows.plain = tab.rows.plain_all = 0;
        tab.chunks = chunks;
        tab.first = tab.it = it;
        tab.it_end = it_end;
    }
    if constexpr (GROUPED) {  // the place among the items in shared memory: kept in registers it spills the sums
        __syncthreads();
        while (tab.it < tab.it_end) {
            it = tab.it;
            const Run run = next_run<NT, GROUPED>(p, tab, tab.chunks, it, tab.it_end);
            if (threadIdx.x == 0) tab.it = it;  // (every thread has read it)
            run_columns<NT, INT>(p, run, tab.rows, smem);
        }
    } else {
        while (it < it_end) {
            const Run run = next_run<NT, GROUPED>(p, tab, chunks, it, it_end);
            run_columns<NT, INT>(p, run, tab.rows, smem);
        }
    }
    if (p.cluster_log ? tab.rows.plain_all : tab.rows.plain) plain_runs<NT, INT, GROUPED>(p, tab);
}

// The clusters of 2^log CTAs that the device holds at once.
template <int NT, bool INT, bool GROUPED>
cudaError_t resident_clusters(int log, int num_sms, int* out) {
    static std::mutex mu;
    static int cache[64][4];
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    if (dev < 0 || dev >= 64) return cudaErrorInvalidDevice;
    if (log == 0) {
        *out = num_sms;
        return cudaSuccess;
    }
    std::lock_guard<std::mutex> lock(mu);
    if (cache[dev][log] == 0) {
        cudaLaunchConfig_t cfg{};
        cfg.gridDim = dim3(unsigned(num_sms >> log << log));
        cfg.blockDim = dim3(kThreads);
        cfg.dynamicSmemBytes = kSmemCap;
        cudaLaunchAttribute attr[1]{};
        attr[0].id = cudaLaunchAttributeClusterDimension;
        attr[0].val.clusterDim.x = 1u << log;
        attr[0].val.clusterDim.y = 1;
        attr[0].val.clusterDim.z = 1;
        cfg.attrs = attr;
        cfg.numAttrs = 1;
        int n = 0;
        e = cudaOccupancyMaxActiveClusters(&n, w4a16_kernel<NT, INT, GROUPED>, &cfg);
        if (e != cudaSuccess) return e;
        if (n < 1) return cudaErrorLaunchOutOfResources;
        cache[dev][log] = n;
    }
    *out = cache[dev][log];
    return cudaSuccess;
}

template <int NT, bool INT, bool GROUPED>
cudaError_t launch_t(Params& p, int num_sms, cudaStream_t stream) {
    constexpr auto kern = w4a16_kernel<NT, INT, GROUPED>;
    constexpr int kRows = rows_of(NT);
    cudaError_t e = configure_once<kern>(kThreads, kSmemCap);
    if (e != cudaSuccess) return e;
    // CTAs that split K: so many that making the tokens' digits stays short, 128
    // (token, block) pairs in a CTA (64 where a pass of 8 tokens is bound by its
    // arithmetic).  K = 11008, N = 4096, 8 tokens: 39.8 us with one CTA, 28.7 with 2,
    // 21.2 with 4, 18.6 with 8; K = 4096, N = 22016: 3 tokens 14.8 with one, 15.7 with 2;
    // 8 tokens 32.2 with one, 22.3 with 2, 20.9 with 4.
    const int nkb = p.K / 128;
    p.max_rows = int(p.R < kRows ? p.R : kRows);
    p.cluster_log = 0;
    const int64_t pairs = int64_t(p.max_rows) * nkb;
    while ((1 << p.cluster_log) < kMaxCluster && pairs > (int64_t(NT == 4 ? 64 : 128) << p.cluster_log) &&
           nkb >= (2 << p.cluster_log))
        ++p.cluster_log;
    const int part = (nkb + (1 << p.cluster_log) - 1) >> p.cluster_log;  // blocks of a CTA, at most
    int clusters = 0;
    if ((e = resident_clusters<NT, INT, GROUPED>(p.cluster_log, num_sms, &clusters)) != cudaSuccess) return e;
    const int64_t live = p.offsets ? (p.E < p.R ? p.E : p.R) : 1;
    const int64_t most = (p.N / 8) * (live + p.R / kRows);  // at most that many items
    if (most < clusters) clusters = int(most);
    // Warps along a CTA's K: all 16, or with fewer blocks than that just enough,
    // the others side by side on tiles of their own.  Fewer warps along K let the
    // sums meet less often: in a cluster at least two blocks a warp, and elsewhere
    // as few as leave six steps (16 tokens, 2 of 8 experts each, K = 4096,
    // N = 14336: 56.3 us with 4 warps, 62.3 with 16).
    p.ks_log = 4;
    while (p.ks_log > 0 && (1 << (p.ks_log - 1)) >= part) --p.ks_log;
    while (p.ks_log > 0 && (part >> p.ks_log) < 2 && p.cluster_log) --p.ks_log;
    const int64_t passes = live > (p.R + kRows - 1) / kRows ? live : (p.R + kRows - 1) / kRows;
    const int64_t cols = p.N * passes / clusters;  // of a cluster, about
    while (p.ks_log > 0 && cols >= 6 * (int64_t(kTileCols * kWarps) >> (p.ks_log - 1))) --p.ks_log;
    // shared memory: the rings, at least one tile's sums, the tokens (panels of
    // K if they do not fit), then more tiles' sums
    const int red = red_bytes(p.max_rows);
    const int64_t want = (int64_t(p.max_rows) * kTokenBytes * part + 15) / 16 * 16;
    p.x_panels = want + kRingBytes + red + (p.cluster_log ? kKeepBytes : 0) > kSmemCap;
    p.keeps = p.x_panels || p.cluster_log;
    const int fixed = kRingBytes + (p.keeps ? kKeepBytes : 0);
    p.x_cap = p.x_panels ? (kSmemCap - fixed - red) / 16 * 16 : int32_t(want);
    p.red_tiles = (kSmemCap - fixed - p.x_cap) / red;
    if (p.red_tiles > kMaxTiles) p.red_tiles = kMaxTiles;
    const int smem = fixed + p.x_cap + p.red_tiles * red;

    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3(unsigned(clusters << p.cluster_log));
    cfg.blockDim = dim3(kThreads);
    cfg.dynamicSmemBytes = size_t(smem);
    cfg.stream = stream;
    cudaLaunchAttribute attr[2]{};
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = 1u << p.cluster_log;
    attr[1].val.clusterDim.y = 1;
    attr[1].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 2;
    return cudaLaunchKernelEx(&cfg, kern, p);
}

template <int NT>
cudaError_t launch_nt(Params& p, bool scale_int, int num_sms, cudaStream_t stream) {
    if (p.offsets)
        return scale_int ? launch_t<NT, true, true>(p, num_sms, stream) : launch_t<NT, false, true>(p, num_sms, stream);
    return scale_int ? launch_t<NT, true, false>(p, num_sms, stream) : launch_t<NT, false, false>(p, num_sms, stream);
}

}  // namespace

cudaError_t launch(Params p, bool scale_int, int num_sms, cudaStream_t stream) {
    // Tokens of a pass: up to 2, 4 or 8, as there are.  An expert's rows are not
    // known here: up to 1.5 or 4.5 an expert on average, passes of 2 or 4 (some
    // experts then take a second one, from L2) beat emptier ones of twice as many
    // (16 tokens, 2 of 8 experts each, K = 4096, N = 14336: 56 us against 94).
    const int64_t live = p.offsets ? (p.E < p.R ? p.E : p.R) : 1;
    if (p.R <= 2 || 2 * p.R <= 3 * live) return launch_nt<1>(p, scale_int, num_sms, stream);
    if (p.R <= 4 || 2 * p.R <= 9 * live) return launch_nt<2>(p, scale_int, num_sms, stream);
    return launch_nt<4>(p, scale_int, num_sms, stream);
}

}  // namespace w4a16
}  // namespace w4a8
