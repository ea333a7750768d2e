// Internal launch entry points of the mixture-of-experts row kernels and of
// the 4-bit-weight products with unquantized tokens (host side).
#pragma once

#include <cuda_runtime.h>

#include <cstdint>

namespace w4a8 {

// Element types of the row kernels and of the W4A16 products.
enum ElemType { kElemF32 = 0, kElemF16 = 1, kElemBf16 = 2 };

namespace moe {

constexpr int kMaxExperts = 256;
constexpr int kMaxTopK = 32;

// Stable sort of n = T * top_k router choices by expert (moe_sort.cu).
struct SortParams {
    const void* ids;       // [n] int32 or int64
    int ids64;
    int32_t n, top_k, E;
    int64_t* offsets;      // [E+1]
    int32_t* row_index;    // [n]
    int32_t* out_row;      // [n]
    int32_t* slot_row;     // [n]
    int* status;
};
cudaError_t launch_sort(const SortParams& p, cudaStream_t stream);

// How a sort of n slots is spread over one cluster of at most `most` CTAs (8, the
// portable number, or 16 where the device can place that many): CTAs, slots of a CTA
// at most, and whether it keeps them in shared memory.
constexpr int32_t kMaxKeptSlots = 24576;
struct SortShape {
    int ctas;
    int32_t per_cta;
    bool keep;
};
constexpr SortShape sort_shape(int32_t n, int most) {
    // one CTA per 1024 slots (4096 slots: 5.4 us, 6.5 with 2048 a CTA; 131072: 15 us
    // with 16 CTAs, 30 with 8)
    int ctas = 1;
    while (ctas < most && int64_t(n) > int64_t(ctas) * 1024) ctas *= 2;
    const int64_t steps = (int64_t(n) + 31) / 32, per_cta = (steps + ctas - 1) / ctas * 32;
    return {ctas, int32_t(per_cta), per_cta <= kMaxKeptSlots};
}

// Rows between token order and expert order (moe_rows.cu).  slot_row NULL:
// slot f's row is row f.
struct RowParams {
    const void* a;            // dispatch: x [T, lda]; combine: y [R, lda]; combine backward: d_out [T, lda]
    const void* b;            // combine backward: y [R, ldb]
    int64_t lda, ldb;         // in elements
    const int32_t* slot_row;  // [T, top_k] or NULL
    const float* weights;     // [T, top_k] or NULL (ones)
    void* out;                // dispatch: x_r [R, H]; combine: out [T, H]; combine backward: d_y [R, H]
    float* d_weights;         // combine backward: [T, top_k]
    int64_t T, R, H;
    int32_t top_k;
    bool zeroed;              // dispatch and combine backward: clear the rows that no slot names
    int* status;
};
cudaError_t launch_dispatch(const RowParams& p, int elem, int num_sms, cudaStream_t stream);
cudaError_t launch_combine(const RowParams& p, int elem_y, int elem_out, int num_sms, cudaStream_t stream);
cudaError_t launch_combine_backward(const RowParams& p, int elem_d, int elem_y, int num_sms, cudaStream_t stream);

}  // namespace moe

namespace w4a16 {

struct Params {
    const void* x;                   // [x_rows, ldx] tokens
    int64_t ldx, x_rows;
    const uint8_t* w;                // packed weights [N, K/2] (one layer), or
    const void* scales;              // its scales [K/group, N]
    const uint8_t* const* w_ptrs;    // E packed weights and
    const void* const* s_ptrs;       // their scales (grouped call)
    const int64_t* offsets;          // [E+1], NULL for one layer
    const int32_t* row_index;        // [R] or NULL
    const int32_t* out_row;          // [R] or NULL
    void* y;                         // [y_rows, N]
    int64_t y_rows, R;
    int32_t E, N, K;
    uint32_t group_magic;            // block kb's group: umulhi(kb, magic), or kb when 0
    int32_t x_type, y_type;          // ElemType
    // 2^8, or 2^8 / alpha for integer scales, in two parts: 1 or less for the tokens,
    // 2 or more for the sums
    float x_scale, out_scale;
    int* status;
    // set by launch(): log2 of the CTAs along K and of the warps along a CTA's
    // part, bytes of shared memory for the tokens, whether that takes panels of
    // K, whether columns' sums are kept, the most tokens of a pass, tiles whose
    // sums meet at a time
    int32_t cluster_log, ks_log, x_cap, x_panels, keeps, max_rows, red_tiles;
};
// scale_int: int16 integer scales, else fp32 ones
cudaError_t launch(Params p, bool scale_int, int num_sms, cudaStream_t stream);

}  // namespace w4a16
}  // namespace w4a8
