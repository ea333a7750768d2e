// Rows between token order and expert order, forward and backward:
//   dispatch           x_r[r(t,s)] = x[t]
//   combine            out[t] = sum_s w[t,s] y[r(t,s)]          (dispatch's gradient with w = 1)
//   combine backward   d_y[r(t,s)] = w[t,s] d_out[t],  d_w[t,s] = <d_out[t], y[r(t,s)]>
// with r(t,s) = slot_row[t,s] (negative: no row; -2 - r: row r is cleared), or
// t * top_k + s without it.
//
// All three are bound by HBM: every kernel is laid out by token, so a token's
// own row is read (or written) once and its top_k routed rows once each, and
// nothing is accumulated through memory: sums are fp32, in slot order, rounded
// once.  No atomics.
//
// Measured at the copy rate's share (2 slots, rows of 8 KB): dispatch 85 %, combine
// 79 %, its gradient 90 %; rows of odd lengths reach 35 to 60 %.
//
// What they need is enough loads in flight: a token's kSlots slots (2 or 4, as
// top_k has) are looked up together, then the loads of all of them go out, U
// pieces each, before the first is used.  Rows whose base, distance and length
// allow it move in pieces of 8 elements (16-byte accesses), others by element.
// (Windows shifted out of two 16-byte accesses for rows of odd lengths were
// tried: their registers cost more than the wider accesses gave.)
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include <atomic>
#include <cstdint>
#include <type_traits>

#include "kernels.h"
#include "moe.h"
#include "sm100_ptx.cuh"

namespace w4a8 {
namespace moe {
namespace {

constexpr int kThreadsLog = 8, kThreads = 1 << kThreadsLog;

// Element i of consecutive elements held in words, as fp32 (bf16: a shift or a mask).
template <typename T>
__device__ __forceinline__ float element(const uint32_t* w, int i) {
    if constexpr (sizeof(T) == 4) {
        return __uint_as_float(w[i]);
    } else if constexpr (std::is_same<T, __nv_bfloat16>::value) {
        return __uint_as_float(i & 1 ? w[i >> 1] & 0xFFFF0000u : w[i >> 1] << 16);
    } else {
        const __half2 h = *reinterpret_cast<const __half2*>(&w[i >> 1]);
        return i & 1 ? __high2float(h) : __low2float(h);
    }
}
// Two values rounded to T, in one word.
template <typename T>
__device__ __forceinline__ uint32_t pair(float lo, float hi) {
    if constexpr (std::is_same<T, __nv_bfloat16>::value) {
        const __nv_bfloat162 h = __floats2bfloat162_rn(lo, hi);
        return *reinterpret_cast<const uint32_t*>(&h);
    } else {
        const __half2 h = __floats2half2_rn(lo, hi);
        return *reinterpret_cast<const uint32_t*>(&h);
    }
}

template <typename T>
__device__ __forceinline__ T from_f(float v);
template <>
__device__ __forceinline__ float from_f<float>(float v) {
    return v;
}
template <>
__device__ __forceinline__ __half from_f<__half>(float v) {
    return __float2half_rn(v);
}
template <>
__device__ __forceinline__ __nv_bfloat16 from_f<__nv_bfloat16>(float v) {
    return __float2bfloat16_rn(v);
}

// E consecutive elements as loaded: E = 8 in 16-byte pieces (16-byte aligned), E = 1 alone.
template <typename T, int E>
struct Piece {
    static constexpr int kWords = E * int(sizeof(T)) / 4 > 0 ? E * int(sizeof(T)) / 4 : 1;
    uint32_t w[kWords];
    __device__ __forceinline__ void load(const T* src) {
        if constexpr (E == 1) {
            if constexpr (sizeof(T) == 4)
                w[0] = __ldg(reinterpret_cast<const uint32_t*>(src));
            else
                w[0] = __ldg(reinterpret_cast<const uint16_t*>(src));
        } else {
#pragma unroll
            for (int i = 0; i < kWords / 4; ++i) {
                const uint4 u = __ldg(reinterpret_cast<const uint4*>(src) + i);
                w[4 * i] = u.x, w[4 * i + 1] = u.y, w[4 * i + 2] = u.z, w[4 * i + 3] = u.w;
            }
        }
    }
    __device__ __forceinline__ float get(int i) const { return element<T>(w, i); }
};

template <typename T, int E>
__device__ __forceinline__ void store_f(T* dst, const float (&v)[E]) {
    if constexpr (E == 1) {
        *dst = from_f<T>(v[0]);
    } else {
        constexpr int kPer = 16 / int(sizeof(T));
#pragma unroll
        for (int i = 0; i < E / kPer; ++i) {
            const float* q = v + i * kPer;
            if constexpr (sizeof(T) == 4)
                reinterpret_cast<uint4*>(dst)[i] = make_uint4(__float_as_uint(q[0]), __float_as_uint(q[1]),
                                                              __float_as_uint(q[2]), __float_as_uint(q[3]));
            else
                reinterpret_cast<uint4*>(dst)[i] = make_uint4(pair<T>(q[0], q[1]), pair<T>(q[2], q[3]),
                                                              pair<T>(q[4], q[5]), pair<T>(q[6], q[7]));
        }
    }
}

// The routed row of slot f: >= 0 a row, -1 none, -2 - r a row r to clear.  A
// row outside [0, R) is none and sets the status word; a row to clear outside is
// none (the caller's rows may end with the last expert's).
__device__ __forceinline__ int32_t slot_target(const RowParams& p, int32_t f) {
    if (!p.slot_row) return f;
    const int32_t v = __ldg(p.slot_row + f);
    if ((v >= 0 ? v : -2 - v) < p.R) return v;
    if (v >= 0) atomicExch(p.status, kStatusInvalidArg);
    return -1;
}

// Rows that no slot names (a slot of -1, or a row outside, leaves one) are known only
// when all slots have been seen.  Where the caller wants them cleared, the grid's
// first CTAs look for them beside the others' work, one CTA for 1024 rows and a share
// of the slots.  While every slot of its share names a row that is all it does: with
// R <= T * top_k distinct rows, one without a slot means a slot without one.  The CTAs
// that find such a slot see by another look at all slots which others do, and share
// the rows: each marks those of its part that are named and clears the rest.  The
// others write named rows only, so nothing has to wait.  (Clearing the whole output
// first would cost a third of a dispatch: 2048 tokens, 2 slots, 8 KB rows.)
constexpr int kClearRows = 1024, kMaxClears = 1024;  // rows of a CTA, CTAs
constexpr int kMarkedRows = 16384;                   // rows marked at a time, at most

unsigned clear_ctas(const RowParams& p) {
    // without slot_row every row of R <= T * top_k is named
    if (!p.zeroed || !p.slot_row) return 0u;
    const int64_t n = (p.R + kClearRows - 1) / kClearRows;
    return unsigned(n < kMaxClears ? n : kMaxClears);
}

// The row that a slot of this value names, 2^31 or more for none.
__device__ __forceinline__ uint32_t named_row(int32_t v) { return uint32_t(v >= 0 ? v : -2 - v); }

template <typename V>
__device__ __noinline__ void clear_unnamed(const int32_t* slot_row, int32_t n, uint32_t R, uint32_t clears, V* out,
                                           int32_t row_len) {
    __shared__ uint32_t named[kMarkedRows / 32];
    __shared__ uint32_t parts[kMaxClears / 32];  // the shares that have a slot without a row
    const uint32_t share = (uint32_t(n) + clears - 1) / clears, own = blockIdx.x * share;
    bool missing = false;
#pragma unroll 4
    for (uint32_t i = threadIdx.x; i < share; i += kThreads)
        if (own + i < uint32_t(n)) missing |= named_row(__ldg(slot_row + own + i)) >= R;
    if (!__syncthreads_or(missing)) return;
    if (threadIdx.x < kMaxClears / 32) parts[threadIdx.x] = 0u;
    __syncthreads();
#pragma unroll 4
    for (int32_t i = threadIdx.x; i < n; i += kThreads)
        if (named_row(__ldg(slot_row + i)) >= R) {
            const uint32_t s = uint32_t(i) / share;
            atomicOr(&parts[s >> 5], 1u << (s & 31u));
        }
    __syncthreads();
    uint32_t before = 0u, all = 0u;
    for (uint32_t w = 0; w < kMaxClears / 32; ++w) {
        all += __popc(parts[w]);
        if (w < blockIdx.x >> 5) before += __popc(parts[w]);
        if (w == blockIdx.x >> 5) before += __popc(parts[w] & ((1u << (blockIdx.x & 31u)) - 1u));
    }
    const uint32_t part = min(((R + all - 1) / all + 31u) & ~31u, uint32_t(kMarkedRows));
    for (uint32_t first = before * part; first < R; first += all * part) {
        const uint32_t rows = min(R - first, part);
        for (uint32_t w = threadIdx.x; w < part / 32; w += kThreads) named[w] = 0u;
        __syncthreads();
#pragma unroll 4
        for (int32_t i = threadIdx.x; i < n; i += kThreads) {
            const uint32_t r = named_row(__ldg(slot_row + i)) - first;
            if (r < rows) atomicOr(&named[r >> 5], 1u << (r & 31u));
        }
        __syncthreads();
        for (uint32_t k = 0; k < rows; k += 32) {
            uint32_t left = ~named[k >> 5];
            if (rows - k < 32u) left &= (1u << (rows - k)) - 1u;
            for (; left; left &= left - 1u) {
                V* row = out + (int64_t(first + k) + __ffs(int(left)) - 1) * row_len;
                for (int32_t c = threadIdx.x; c < row_len; c += kThreads) row[c] = V{};
            }
        }
        __syncthreads();
    }
}

// Item g of the grid: a CTA's tokens, `tpt` threads each (a power of two, 32 to
// 256), and, for the kernels whose columns are independent, one of `chunks`
// column ranges.
struct Place {
    int32_t token;  // T or more: none
    int32_t chunk;
};
__device__ __forceinline__ Place place(const RowParams& p, uint32_t g, int tpt_log, uint32_t chunks) {
    Place q;
    q.chunk = 0;
    if (chunks > 1) {
        const uint32_t t = g / chunks;
        q.chunk = int32_t(g - t * chunks);
        g = t;
    }
    q.token = int32_t((g << (kThreadsLog - tpt_log)) + (threadIdx.x >> tpt_log));
    return q;
}

// ---- dispatch: a copy, V the unit (16 bytes, or one element when rows are not
// 16-byte aligned), one item per CTA; eight CTAs an SM (with 34 registers instead of
// 32 there are six: 9.4 us against 9.2)
template <typename V, int U, int kLog>
__global__ void __launch_bounds__(kThreads, 8) dispatch_kernel(const RowParams p, int32_t nv, int64_t ldv, int tpt_log_,
                                                            uint32_t chunks, uint32_t clears) {
    const int tpt_log = kLog > 0 ? kLog : tpt_log_;
    griddep_wait();  // x and slot_row may be the previous kernel's output, x_r its input
    if (threadIdx.x == 0) griddep_launch_dependents();
    if (blockIdx.x < clears) {
        clear_unnamed(p.slot_row, int32_t(p.T * p.top_k), uint32_t(p.R), clears, static_cast<V*>(p.out), nv);
        return;
    }
    const int tpt = 1 << tpt_log, lane = threadIdx.x & (tpt - 1);
    V* dst = static_cast<V*>(p.out);
    const Place q = place(p, blockIdx.x - clears, tpt_log, chunks);
    if (q.token >= p.T) return;
    const V* src = static_cast<const V*>(p.a) + q.token * ldv;
    const int32_t f0 = q.token * p.top_k;
    for (int32_t c = q.chunk * tpt * U + lane; c < nv; c += int32_t(chunks) * tpt * U) {
        V v[U];
#pragma unroll
        for (int u = 0; u < U; ++u)
            if (c + u * tpt < nv) v[u] = __ldg(src + c + u * tpt);
        for (int s = 0; s < p.top_k; ++s) {
            const int32_t r = slot_target(p, f0 + s);
            if (r == -1) continue;
            V* row = dst + int64_t(r >= 0 ? r : -2 - r) * nv;
#pragma unroll
            for (int u = 0; u < U; ++u)
                if (c + u * tpt < nv) row[c + u * tpt] = r >= 0 ? v[u] : V{};
        }
    }
}

// ---- combine: E elements a piece, U pieces of kSlots slots in flight; the next
// item's slots are looked up while this one's rows are on their way
template <typename TY, typename TO, int E, int U, int kSlots, int kLog>
__global__ void __launch_bounds__(kThreads) combine_kernel(const RowParams p, int tpt_log_, uint32_t chunks,
                                                           uint32_t items) {
    const int tpt_log = kLog > 0 ? kLog : tpt_log_;
    griddep_wait();  // y, weights and slot_row may be the previous kernel's output, out its input
    if (threadIdx.x == 0) griddep_launch_dependents();
    const int tpt = 1 << tpt_log, lane = threadIdx.x & (tpt - 1);
    const TY* y = static_cast<const TY*>(p.a);
    const int32_t nv = int32_t(p.H / E);
    struct Slots {
        int32_t r[kSlots];
        float w[kSlots];
    };
    const auto look_up = [&](int32_t token, int s0, Slots& s) {
#pragma unroll
        for (int i = 0; i < kSlots; ++i) {
            s.r[i] = -1;
            s.w[i] = 1.0f;
            if (token < p.T && s0 + i < p.top_k) {
                s.r[i] = slot_target(p, token * p.top_k + s0 + i);
                if (p.weights) s.w[i] = __ldg(p.weights + token * p.top_k + s0 + i);
            }
        }
    };
    uint32_t g = blockIdx.x;
    Slots next;
    look_up(place(p, g, tpt_log, chunks).token, 0, next);
    for (; g < items; g += gridDim.x) {
        const Place q = place(p, g, tpt_log, chunks);
        Slots s = next;
        if (g + gridDim.x < items) look_up(place(p, g + gridDim.x, tpt_log, chunks).token, 0, next);
        if (q.token >= p.T) continue;
        TO* out = static_cast<TO*>(p.out) + q.token * p.H;
        for (int32_t c = q.chunk * tpt * U + lane; c < nv; c += int32_t(chunks) * tpt * U) {
            float acc[U][E];
#pragma unroll
            for (int u = 0; u < U; ++u)
#pragma unroll
                for (int j = 0; j < E; ++j) acc[u][j] = 0.0f;
            for (int s0 = 0; s0 < p.top_k; s0 += kSlots) {
                if (p.top_k > kSlots) look_up(q.token, s0, s);
                Piece<TY, E> v[kSlots][U];
#pragma unroll
                for (int i = 0; i < kSlots; ++i)
                    if (s.r[i] >= 0)
#pragma unroll
                        for (int u = 0; u < U; ++u)
                            if (c + u * tpt < nv) v[i][u].load(y + s.r[i] * p.lda + (c + u * tpt) * E);
#pragma unroll
                for (int i = 0; i < kSlots; ++i)
                    if (s.r[i] >= 0)
#pragma unroll
                        for (int u = 0; u < U; ++u)
#pragma unroll
                            for (int j = 0; j < E; ++j) acc[u][j] = __fmaf_rn(s.w[i], v[i][u].get(j), acc[u][j]);
            }
#pragma unroll
            for (int u = 0; u < U; ++u)
                if (c + u * tpt < nv) store_f<TO, E>(out + (c + u * tpt) * E, acc[u]);
        }
    }
}

// ---- combine backward: kSlots slots at a time share the pieces of d_out[t]
template <typename TD, typename TY, int E, int U, int kSlots, int kLog>
__global__ void __launch_bounds__(kThreads) combine_backward_kernel(const RowParams p, int tpt_log_, uint32_t items,
                                                                    uint32_t clears) {
    const int tpt_log = kLog > 0 ? kLog : tpt_log_;
    __shared__ float red[kThreads / 32][kSlots];
    griddep_wait();  // the inputs may be the previous kernel's output, d_y and d_weights its input
    if (threadIdx.x == 0) griddep_launch_dependents();
    const int tpt = 1 << tpt_log, lane = threadIdx.x & (tpt - 1), warp = threadIdx.x >> 5;
    const TY* y = static_cast<const TY*>(p.b);
    TY* d_y = static_cast<TY*>(p.out);
    if (blockIdx.x < clears) {
        // whole words where the rows are known to be aligned
        using V = std::conditional_t<E == 1, std::conditional_t<sizeof(TY) == 4, uint32_t, uint16_t>, uint4>;
        clear_unnamed(p.slot_row, int32_t(p.T * p.top_k), uint32_t(p.R), clears, reinterpret_cast<V*>(d_y),
                      int32_t(p.H * sizeof(TY) / sizeof(V)));
        return;
    }
    for (uint32_t g = blockIdx.x - clears; g < items; g += gridDim.x - clears) {
        const int32_t token = place(p, g, tpt_log, 1).token;
        const bool live = token < p.T;
        const TD* d = static_cast<const TD*>(p.a) + (live ? token : 0) * p.lda;
        const int32_t f0 = (live ? token : 0) * p.top_k;
        const int32_t nv = live ? int32_t(p.H / E) : 0;
        for (int s0 = 0; s0 < p.top_k; s0 += kSlots) {
            int32_t r[kSlots];
            float w[kSlots], dot[kSlots];
#pragma unroll
            for (int i = 0; i < kSlots; ++i) {
                const bool in = live && s0 + i < p.top_k;
                r[i] = in ? slot_target(p, f0 + s0 + i) : -1;
                w[i] = in ? __ldg(p.weights + f0 + s0 + i) : 0.0f;
                dot[i] = 0.0f;
            }
            for (int32_t c = lane; c < nv; c += tpt * U) {
                Piece<TD, E> dv[U];
                Piece<TY, E> yv[kSlots][U];
#pragma unroll
                for (int u = 0; u < U; ++u)
                    if (c + u * tpt < nv) dv[u].load(d + (c + u * tpt) * E);
#pragma unroll
                for (int i = 0; i < kSlots; ++i)
                    if (r[i] >= 0)
#pragma unroll
                        for (int u = 0; u < U; ++u)
                            if (c + u * tpt < nv) yv[i][u].load(y + r[i] * p.ldb + (c + u * tpt) * E);
#pragma unroll
                for (int i = 0; i < kSlots; ++i) {
                    if (r[i] == -1) continue;
                    TY* row = d_y + (r[i] >= 0 ? r[i] : -2 - r[i]) * p.H;
#pragma unroll
                    for (int u = 0; u < U; ++u) {
                        if (c + u * tpt >= nv) continue;
                        float v[E];
#pragma unroll
                        for (int j = 0; j < E; ++j) {
                            v[j] = 0.0f;
                            if (r[i] >= 0) {
                                dot[i] = __fmaf_rn(dv[u].get(j), yv[i][u].get(j), dot[i]);
                                v[j] = __fmul_rn(w[i], dv[u].get(j));
                            }
                        }
                        store_f<TY, E>(row + (c + u * tpt) * E, v);
                    }
                }
            }
#pragma unroll
            for (int i = 0; i < kSlots; ++i) {
#pragma unroll
                for (int o = 16; o > 0; o >>= 1) dot[i] += __shfl_xor_sync(0xffffffffu, dot[i], o);
                if ((threadIdx.x & 31) == 0) red[warp][i] = dot[i];
            }
            __syncthreads();
            if (live && lane < kSlots && s0 + lane < p.top_k) {
                float sum = 0.0f;
                for (int i = 0; i < tpt / 32; ++i) sum += red[warp + i][lane];
                p.d_weights[f0 + s0 + lane] = sum;
            }
            __syncthreads();
        }
    }
}

// The launch of a row kernel: threads per token, enough that a token's pieces
// are covered once by U a thread (32 to 256); column ranges per token, so that a
// few tokens still fill the GPU, no more than the row has steps; a grid of the
// CTAs that the device holds at once.
struct Shape {
    int tpt_log = 5;
    uint32_t chunks = 1, items = 0;
    unsigned grid = 0;
};
template <auto kern>
cudaError_t shape_of(int64_t pieces, int U, int64_t T, bool split, int num_sms, Shape* s, int log = 0) {
    static std::atomic<int> resident[64];
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    if (dev < 0 || dev >= 64) return cudaErrorInvalidDevice;
    int per_sm = resident[dev].load();
    if (per_sm == 0) {
        e = cudaOccupancyMaxActiveBlocksPerMultiprocessor(&per_sm, kern, kThreads, 0);
        if (e != cudaSuccess) return e;
        if (per_sm < 1) per_sm = 1;
        resident[dev].store(per_sm);
    }
    if (log > 0) s->tpt_log = log;
    while (log == 0 && s->tpt_log < kThreadsLog && (int64_t(U) << s->tpt_log) < pieces) ++s->tpt_log;
    const int64_t per_cta = int64_t(1) << (kThreadsLog - s->tpt_log), groups = (T + per_cta - 1) / per_cta;
    if (split) {
        const int64_t steps = (pieces + (int64_t(U) << s->tpt_log) - 1) / (int64_t(U) << s->tpt_log);
        int64_t want = (2 * int64_t(num_sms) + groups - 1) / groups;
        if (want > steps) want = steps;
        if (want > 1) s->chunks = uint32_t(want);
    }
    const int64_t items = groups * s->chunks, most = int64_t(num_sms) * per_sm;
    if (items + most > INT32_MAX) return cudaErrorInvalidValue;
    s->items = uint32_t(items);
    s->grid = unsigned(items < most ? items : most);
    return cudaSuccess;
}

bool aligned(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

template <typename V, int U, int kLog>
cudaError_t dispatch_t(const RowParams& p, int64_t nv, int64_t ldv, int num_sms, cudaStream_t stream) {
    Shape s;
    constexpr auto kern = dispatch_kernel<V, U, kLog>;
    const cudaError_t e = shape_of<kern>(nv, U, p.T, true, num_sms, &s, kLog);
    if (e != cudaSuccess) return e;
    // not the CTAs that the device holds at once: one per item was faster (14.3
    // against 16.0 us, 2048 tokens, 8 slots, rows of 4 KB)
    const unsigned clears = clear_ctas(p);
    const LaunchPdl lc(s.items + clears, kThreads, 0, stream);
    return cudaLaunchKernelEx(&lc.cfg, kern, p, int32_t(nv), ldv, s.tpt_log, s.chunks, clears);
}

template <typename TY, typename TO, int E, int U, int kSlots, int kLog>
cudaError_t combine_e(const RowParams& p, int num_sms, cudaStream_t stream) {
    Shape s;
    constexpr auto kern = combine_kernel<TY, TO, E, U, kSlots, kLog>;
    const cudaError_t e = shape_of<kern>(p.H / E, U, p.T, true, num_sms, &s, kLog);
    if (e != cudaSuccess) return e;
    const LaunchPdl lc(s.grid, kThreads, 0, stream);
    return cudaLaunchKernelEx(&lc.cfg, kern, p, s.tpt_log, s.chunks, s.items);
}

// Two slots of many long 16-bit rows take 128 threads a token with two pieces of each
// slot in flight, else 256 threads and one.  The rule, measured at 150 to 8192 tokens and
// rows of 1024 to 14336 (148 SMs): combine gains 2 to 14 % from 1600 tokens of 2048 on
// (4096 tokens of 4096: 20.5 us against 21.9) and loses 1 to 11 % at 592 and 1200 (1200
// of 8192: 15.8 against 14.2); rows of 1024 lose 21 %.  The gradient gains 2 to 10 % up to
// rows of 4096 (4096 tokens: 29.4 against 30.6) and loses 1 to 7 % with longer ones
// (8192 tokens of 8192: 114 against 107).  fp32 rows and more slots lose by it (18.7
// against 18.4, 20.9 against 19.6).
bool many_long_rows(const RowParams& p, size_t elem_bytes, int num_sms) {
    return elem_bytes == 2 && p.top_k <= 2 && p.H >= 2048 && p.T >= 10 * int64_t(num_sms);
}

// Rows in 16-byte pieces of 8 elements (both types): lengths a multiple of 8,
// bases and strides 16-byte aligned.  Otherwise one element at a time, with the
// threads per token (32 or 256) known at compile time: the pieces of a thread are then
// constant distances apart, which halves the registers (2048 tokens, 2 slots, 4095
// bf16: 15.8 us against 22.0).
template <typename TY, typename TO>
cudaError_t combine_t(const RowParams& p, int num_sms, cudaStream_t stream) {
    const bool two = p.top_k <= 2, shorter = p.H < 1024;
    const bool many = many_long_rows(p, sizeof(TY), num_sms);
    if (p.H % 8 == 0 && aligned(p.a) && aligned(p.out) && p.lda * int64_t(sizeof(TY)) % 16 == 0)
        return many  ? combine_e<TY, TO, 8, 2, 2, 7>(p, num_sms, stream)
               : two ? combine_e<TY, TO, 8, 1, 2, 0>(p, num_sms, stream)
                     : combine_e<TY, TO, 8, 1, 4, 0>(p, num_sms, stream);
    if (shorter)
        return two ? combine_e<TY, TO, 1, 8, 2, 5>(p, num_sms, stream) : combine_e<TY, TO, 1, 4, 4, 5>(p, num_sms, stream);
    return two ? combine_e<TY, TO, 1, 8, 2, 8>(p, num_sms, stream) : combine_e<TY, TO, 1, 4, 4, 8>(p, num_sms, stream);
}

template <typename TD, typename TY, int E, int U, int kSlots, int kLog>
cudaError_t backward_e(const RowParams& p, int num_sms, cudaStream_t stream) {
    Shape s;
    constexpr auto kern = combine_backward_kernel<TD, TY, E, U, kSlots, kLog>;
    const cudaError_t e = shape_of<kern>(p.H / E, U, p.T, false, num_sms, &s, kLog);
    if (e != cudaSuccess) return e;
    // the clearing CTAs take the place of others that the device would hold at once
    const unsigned clears = clear_ctas(p);
    unsigned grid = s.grid;
    if (grid < s.items) grid = grid > 2 * clears ? grid - clears : grid / 2;
    const LaunchPdl lc(grid + clears, kThreads, 0, stream);
    return cudaLaunchKernelEx(&lc.cfg, kern, p, s.tpt_log, s.items, clears);
}

template <typename TD, typename TY>
cudaError_t backward_t(const RowParams& p, int num_sms, cudaStream_t stream) {
    const bool two = p.top_k <= 2, shorter = p.H < 1024;
    const bool many = many_long_rows(p, sizeof(TY), num_sms) && p.H <= 4096;
    if (p.H % 8 == 0 && aligned(p.a) && aligned(p.b) && aligned(p.out) && p.lda * int64_t(sizeof(TD)) % 16 == 0 &&
        p.ldb * int64_t(sizeof(TY)) % 16 == 0)
        return many  ? backward_e<TD, TY, 8, 2, 2, 7>(p, num_sms, stream)
               : two ? backward_e<TD, TY, 8, 1, 2, 0>(p, num_sms, stream)
                     : backward_e<TD, TY, 8, 1, 4, 0>(p, num_sms, stream);
    if (shorter)
        return two ? backward_e<TD, TY, 1, 4, 2, 5>(p, num_sms, stream) : backward_e<TD, TY, 1, 4, 4, 5>(p, num_sms, stream);
    return two ? backward_e<TD, TY, 1, 4, 2, 8>(p, num_sms, stream) : backward_e<TD, TY, 1, 4, 4, 8>(p, num_sms, stream);
}

// Calls f with a value of the element type (a tag).
template <typename F>
cudaError_t with_type(int elem, F&& f) {
    if (elem == kElemF32) return f(float{});
    if (elem == kElemF16) return f(__half{});
    return f(__nv_bfloat16{});
}

}  // namespace

cudaError_t launch_dispatch(const RowParams& p, int elem, int num_sms, cudaStream_t stream) {
    const int64_t esz = elem == kElemF32 ? 4 : 2;
    if (p.H * esz % 16 == 0 && p.lda * esz % 16 == 0 && aligned(p.a) && aligned(p.out))
        return dispatch_t<uint4, 2, 0>(p, p.H * esz / 16, p.lda * esz / 16, num_sms, stream);
    // by element, as in combine_t
    if (p.H < 1024)
        return esz == 4 ? dispatch_t<uint32_t, 8, 5>(p, p.H, p.lda, num_sms, stream)
                        : dispatch_t<uint16_t, 8, 5>(p, p.H, p.lda, num_sms, stream);
    return esz == 4 ? dispatch_t<uint32_t, 8, 8>(p, p.H, p.lda, num_sms, stream)
                    : dispatch_t<uint16_t, 8, 8>(p, p.H, p.lda, num_sms, stream);
}

cudaError_t launch_combine(const RowParams& p, int elem_y, int elem_out, int num_sms, cudaStream_t stream) {
    return with_type(elem_y, [&](auto ty) {
        return with_type(elem_out, [&](auto to) {
            return combine_t<decltype(ty), decltype(to)>(p, num_sms, stream);
        });
    });
}

cudaError_t launch_combine_backward(const RowParams& p, int elem_d, int elem_y, int num_sms, cudaStream_t stream) {
    return with_type(elem_d, [&](auto td) {
        return with_type(elem_y, [&](auto ty) { return backward_t<decltype(td), decltype(ty)>(p, num_sms, stream); });
    });
}

}  // namespace moe
}  // namespace w4a8
