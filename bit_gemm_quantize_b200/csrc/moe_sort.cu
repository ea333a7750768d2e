// Router choices sorted by expert: a stable counting sort of the n = T * top_k
// slots, on the device, so that the routed-order quantizer, the row kernels and
// the grouped products can follow in the stream with no host round trip.
//   offsets[e] = #{f : id[f] < e},  r(f) = offsets[id[f]] + #{f' < f : id[f'] = id[f]}
// Slots that name no expert form one more bin behind the last expert's.
//
// Bound by latency: the bytes (4 or 8 read and 12 written a slot) are nothing
// against the steps in a row, so there is one launch, by one cluster of CTAs.
// Every warp owns a contiguous piece of the slots and counts it into a row of
// its own in shared memory (one lane adds for all equal ones, found by a vote on
// each bit of the bin: match_any costs as much as 32 different values are, 300
// cycles a step measured at 256 experts); one
// pass over the warps' rows and one over the cluster's CTAs (distributed shared
// memory) turn the counts into every warp's first row per bin, and the warps
// walk their pieces again.  No atomics, so the order is the same in every run;
// the cluster barrier is the only wait.
//
// A CTA keeps its slots' marks (bin and rank) and their sorted order in shared memory, so that
// ids are read once and the rows of a bin are written side by side: written one
// by one in slot order they are 4-byte stores to as many sectors.  Pieces too
// long for shared memory are read twice and written one by one.
#include <cooperative_groups.h>
#include <cuda_runtime.h>

#include <atomic>
#include <cstdint>

#include "kernels.h"
#include "moe.h"
#include "sm100_ptx.cuh"

namespace w4a8 {
namespace moe {
namespace {

namespace cg = cooperative_groups;

constexpr int kSortThreads = 1024;
constexpr int kSortWarps = kSortThreads / 32;
constexpr int kBinsMax = kMaxExperts + 1;
constexpr int kBatch = 8;             // ids in flight per lane
constexpr int kSlotBytes = 6;         // a slot's place in the sorted order and its mark

template <typename ID>
__device__ __forceinline__ int bin_of(ID id, int32_t E, bool& bad) {
    if (id >= 0 && id < ID(E)) return int(id);
    bad |= id != ID(-1);
    return E;
}

// The lanes whose bin equals this lane's (0 for a lane without a slot, bin -1).
__device__ __forceinline__ unsigned lanes_of(int bin, int bits) {
    unsigned same = __ballot_sync(0xffffffffu, bin >= 0);
    for (int i = 0; i < bits; ++i) {
        const unsigned set = __ballot_sync(0xffffffffu, (bin >> i) & 1);
        same &= (bin >> i) & 1 ? set : ~set;
    }
    return bin >= 0 ? same : 0u;
}

// The bins of the slots f0 + 32 i + lane, i < kBatch (-1 from `end` on).
template <typename ID>
__device__ __forceinline__ void load_bins(const ID* ids, int64_t f0, int64_t end, int32_t E, bool& bad,
                                          int (&bin)[kBatch]) {
    ID id[kBatch];
#pragma unroll
    for (int i = 0; i < kBatch; ++i) {
        const int64_t f = f0 + 32 * i + (threadIdx.x & 31);
        id[i] = f < end ? ids[f] : ID(-1);
    }
#pragma unroll
    for (int i = 0; i < kBatch; ++i) {
        const int64_t f = f0 + 32 * i + (threadIdx.x & 31);
        bin[i] = f < end ? bin_of(id[i], E, bad) : -1;
    }
}

// KEEP: the CTA's slots are kept in shared memory.
template <typename ID, bool KEEP>
__global__ void __launch_bounds__(kSortThreads) sort_kernel(const SortParams p, int32_t kept_cap) {
    extern __shared__ int32_t dyn[];
    __shared__ int32_t hist[kSortWarps][kBinsMax];
    __shared__ int32_t total[kBinsMax];
    __shared__ int32_t base[kBinsMax];   // first row of the CTA's slots of a bin
    __shared__ int32_t local[kBinsMax];  // and their first place in the CTA's own order
    __shared__ int32_t warp_sum[2][kSortWarps];
    int32_t* order = dyn;                                          // [kept_cap]: slot (within the CTA) by place
    // [kept_cap], by slot: its bin (9 bits), how many lanes of its step come before
    // it in the bin (5) and whether it is the last of them
    uint16_t* mark_s = reinterpret_cast<uint16_t*>(dyn + kept_cap);
    cg::cluster_group cluster = cg::this_cluster();
    const int C = int(cluster.num_blocks()), rank = int(cluster.block_rank());
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const unsigned below = (1u << lane) - 1u;
    const int bins = p.E + 1, bits = 32 - __clz(p.E);
    const ID* ids = static_cast<const ID*>(p.ids);
    for (int i = threadIdx.x; i < kSortWarps * kBinsMax; i += kSortThreads) (&hist[0][0])[i] = 0;
    griddep_wait();  // the ids may be the previous kernel's output, the outputs its input
    if (threadIdx.x == 0) griddep_launch_dependents();
    __syncthreads();

    // the CTA's and this warp's pieces: whole steps of 32 slots, in order
    const int64_t steps = (int64_t(p.n) + 31) / 32;
    const int64_t c0 = steps * rank / C, c1 = steps * (rank + 1) / C;
    const int64_t f_cta = c0 * 32;
    const int64_t f0 = (c0 + (c1 - c0) * warp / kSortWarps) * 32;
    const int64_t f1 = min((c0 + (c1 - c0) * (warp + 1) / kSortWarps) * 32, int64_t(p.n));
    bool bad = false;
    for (int64_t f = f0; f < f1; f += 32 * kBatch) {
        int bin[kBatch];
        load_bins(ids, f, f1, p.E, bad, bin);
#pragma unroll
        for (int i = 0; i < kBatch; ++i) {
            if (f + 32 * i >= f1) break;
            const unsigned same = lanes_of(bin[i], bits);
            if (bin[i] >= 0) {
                const int rank = __popc(same & below);
                const bool last = same >> lane == 1u;
                if (last) hist[warp][bin[i]] += rank + 1;
                if constexpr (KEEP) mark_s[f + 32 * i + lane - f_cta] = uint16_t(bin[i] | rank << 9 | int(last) << 14);
            }
            __syncwarp();
        }
    }
    if (bad) atomicExch(p.status, kStatusInvalidArg);
    __syncthreads();

    // counts -> exclusive prefix over the CTA's warps, and the CTA's totals
    const int b = threadIdx.x;
    int32_t mine = 0;
    if (b < bins) {
        int32_t c[kSortWarps];
#pragma unroll
        for (int i = 0; i < kSortWarps; ++i) c[i] = hist[i][b];
#pragma unroll
        for (int i = 0; i < kSortWarps; ++i) {
            hist[i][b] = mine;
            mine += c[i];
        }
        total[b] = mine;
    }
    cluster.sync();
    int32_t before = 0, all = 0;
    if (b < bins) {
        for (int c = 0; c < C; ++c) {
            const int32_t v = cluster.map_shared_rank(total, c)[b];
            all += v;
            if (c < rank) before += v;
        }
    }
    // exclusive scans over the bins (one per thread): all slots, and the CTA's own
    int32_t incl = all, own = mine;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int32_t v = __shfl_up_sync(0xffffffffu, incl, o), u = __shfl_up_sync(0xffffffffu, own, o);
        if (lane >= o) {
            incl += v;
            own += u;
        }
    }
    if (lane == 31) {
        warp_sum[0][warp] = incl;
        warp_sum[1][warp] = own;
    }
    __syncthreads();
    if (b < bins) {
        int32_t first = incl - all, place = own - mine;
        for (int i = 0; i < warp; ++i) {
            first += warp_sum[0][i];
            place += warp_sum[1][i];
        }
        base[b] = first + before;
        local[b] = place;
        if (rank == 0) p.offsets[b] = first;  // bin E: the slots kept
    }
    cluster.sync();  // no CTA leaves while another reads its totals; base and local are complete

    const uint32_t k = uint32_t(p.top_k);
    const auto place = [&](int64_t f, int bin, int rank, bool last) {  // the slots of a step, f of this lane
        int32_t at = 0;                                                // among the CTA's slots of the bin
        if (bin >= 0) at = hist[warp][bin] + rank;
        __syncwarp();  // every lane has read its count
        if (bin >= 0) {
            if (last) hist[warp][bin] = at + 1;
            const int32_t r = base[bin] + at;
            const bool kept = bin < p.E;
            p.slot_row[f] = kept ? r : -2 - r;
            if constexpr (KEEP) {
                order[local[bin] + at] = int32_t(f - f_cta);
            } else {
                p.row_index[r] = kept ? int32_t(uint32_t(f) / k) : -1;
                p.out_row[r] = kept ? int32_t(f) : -1;
            }
        }
        __syncwarp();
    };
    if constexpr (KEEP) {
        for (int64_t f = f0 + lane; f - lane < f1; f += 32) {
            const int m = f < f1 ? mark_s[f - f_cta] : -1;
            place(f, m < 0 ? -1 : m & 511, (m >> 9) & 31, m >> 14 & 1);
        }
    } else {
        for (int64_t f = f0; f < f1; f += 32 * kBatch) {
            int bin[kBatch];
            load_bins(ids, f, f1, p.E, bad, bin);
#pragma unroll
            for (int i = 0; i < kBatch; ++i) {
                if (f + 32 * i >= f1) break;
                const unsigned same = lanes_of(bin[i], bits);
                place(f + 32 * i + lane, bin[i], __popc(same & below), same >> lane == 1u);
            }
        }
    }
    if constexpr (KEEP) {
        __syncthreads();
        const int32_t n_cta = int32_t(min(c1 * 32, int64_t(p.n)) - f_cta);
        for (int32_t i = threadIdx.x; i < n_cta; i += kSortThreads) {
            const int32_t fl = order[i], bin = mark_s[fl] & 511;
            const int32_t r = base[bin] + (i - local[bin]);
            const int32_t f = int32_t(f_cta) + fl;
            const bool kept = bin < p.E;
            p.row_index[r] = kept ? int32_t(uint32_t(f) / k) : -1;
            p.out_row[r] = kept ? f : -1;
        }
    }
}

// The launch of a cluster of C CTAs.
struct LaunchCluster {
    cudaLaunchConfig_t cfg{};
    cudaLaunchAttribute attr[2]{};
    LaunchCluster(int C, size_t smem, cudaStream_t stream) {
        cfg.gridDim = dim3(unsigned(C));
        cfg.blockDim = dim3(kSortThreads);
        cfg.dynamicSmemBytes = smem;
        cfg.stream = stream;
        attr[0].id = cudaLaunchAttributeClusterDimension;
        attr[0].val.clusterDim.x = unsigned(C);
        attr[0].val.clusterDim.y = 1;
        attr[0].val.clusterDim.z = 1;
        attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
        attr[1].val.programmaticStreamSerializationAllowed = 1;
        cfg.attrs = attr;
        cfg.numAttrs = 2;
    }
    LaunchCluster(const LaunchCluster&) = delete;
    LaunchCluster& operator=(const LaunchCluster&) = delete;
};

template <typename ID, bool KEEP>
cudaError_t launch_t(const SortParams& p, const SortShape& shape, cudaStream_t stream) {
    const cudaError_t e = configure_once<sort_kernel<ID, KEEP>>(kSortThreads, kMaxKeptSlots * kSlotBytes);
    if (e != cudaSuccess) return e;
    const LaunchCluster lc(shape.ctas, KEEP ? size_t(shape.per_cta) * kSlotBytes : 0, stream);
    return cudaLaunchKernelEx(&lc.cfg, sort_kernel<ID, KEEP>, p, shape.per_cta);
}

// The most CTAs of a cluster on the current device: 16, more than the portable eight,
// if it can place them at all (a partition with small GPCs may not).
template <typename ID>
cudaError_t most_ctas(int* out) {
    static std::atomic<int> known[64];
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    if (dev < 0 || dev >= 64) return cudaErrorInvalidDevice;
    *out = known[dev].load();
    if (*out != 0) return cudaSuccess;
    *out = 16;
    const auto ask = [&](auto kern, int smem) {
        if (*out < 16) return;
        cudaError_t r = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
        if (r == cudaSuccess) r = cudaFuncSetAttribute(kern, cudaFuncAttributeNonPortableClusterSizeAllowed, 1);
        const LaunchCluster lc(16, size_t(smem), nullptr);
        int n = 0;
        if (r == cudaSuccess) r = cudaOccupancyMaxActiveClusters(&n, kern, &lc.cfg);
        if (r != cudaSuccess || n < 1) {
            *out = 8;
            cudaGetLastError();  // not a failure of the call
        }
    };
    ask(sort_kernel<ID, true>, kMaxKeptSlots * kSlotBytes);
    ask(sort_kernel<ID, false>, kMaxKeptSlots * kSlotBytes);
    known[dev].store(*out);
    return cudaSuccess;
}

template <typename ID>
cudaError_t launch_id(const SortParams& p, cudaStream_t stream) {
    int most = 8;
    if (sort_shape(p.n, 16).ctas > 8) {
        const cudaError_t e = most_ctas<ID>(&most);
        if (e != cudaSuccess) return e;
    }
    const SortShape shape = sort_shape(p.n, most);
    return shape.keep ? launch_t<ID, true>(p, shape, stream) : launch_t<ID, false>(p, shape, stream);
}

}  // namespace

cudaError_t launch_sort(const SortParams& p, cudaStream_t stream) {
    return p.ids64 ? launch_id<int64_t>(p, stream) : launch_id<int32_t>(p, stream);
}

}  // namespace moe
}  // namespace w4a8
