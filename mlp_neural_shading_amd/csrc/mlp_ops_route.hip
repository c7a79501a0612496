// mlp_ops_route.hip -- the router's choice of experts, and the order of rows by expert.
#include <hip/hip_runtime.h>

#include "mlp_ops_kernels.h"

namespace mlpk {

namespace {

// ---- the router --------------------------------------------------------------------------------

constexpr double kNone = -__builtin_huge_val();  // the choice of an expert that cannot be chosen

__device__ __forceinline__ double wave_max(double v)
{
#pragma unroll
    for (int d = 32; d; d >>= 1)
        v = fmax(v, __shfl_xor(v, d));
    return v;
}

__device__ __forceinline__ double wave_sum(double v)
{
#pragma unroll
    for (int d = 32; d; d >>= 1)
        v += __shfl_xor(v, d);
    return v;
}

// The largest value and the lowest index that has it, over the wave.
__device__ __forceinline__ void wave_argmax(double &v, int &i)
{
#pragma unroll
    for (int d = 32; d; d >>= 1) {
        const double ov = __shfl_xor(v, d);
        const int oi = __shfl_xor(i, d);
        if (ov > v || (ov == v && oi < i)) {
            v = ov;
            i = oi;
        }
    }
}

// One wave per token; lane l holds the experts l, l + 64, ...  Scores and choices in 64 bits: two experts'
// choices may lie closer together than FP32 tells apart.
template <class T, int VPL>
__global__ __launch_bounds__(64) void route_tokens(RouteArgs r)
{
    extern __shared__ double choice_lds[];  // [experts] choices, then [groups] group values
    const int lane = threadIdx.x;
    for (int64_t t = blockIdx.x; t < r.tokens; t += gridDim.x) {
        const T *x = (const T *)r.logits + t * r.ld;
        double score[VPL], choice[VPL];
        bool open[VPL];
        double m = kNone;
#pragma unroll
        for (int v = 0; v < VPL; ++v) {
            const int e = v * 64 + lane;
            score[v] = e < r.experts ? (double)(float)x[e] : kNone;
            open[v] = score[v] > kNone;  // neither NaN nor -infinity
            m = open[v] ? fmax(m, score[v]) : m;
        }
        if (r.sigmoid) {
#pragma unroll
            for (int v = 0; v < VPL; ++v)
                score[v] = open[v] ? 1.0 / (1.0 + exp(-score[v])) : 0.0;
        } else {
            m = wave_max(m);
            double sum = 0.0;
#pragma unroll
            for (int v = 0; v < VPL; ++v) {
                score[v] = !open[v] ? 0.0 : score[v] == m ? 1.0 : exp(score[v] - m);  // of infinities too
                sum += score[v];
            }
            sum = wave_sum(sum);
#pragma unroll
            for (int v = 0; v < VPL; ++v)
                score[v] = open[v] ? score[v] / sum : 0.0;
        }
#pragma unroll
        for (int v = 0; v < VPL; ++v) {
            const int e = v * 64 + lane;
            choice[v] = open[v] ? score[v] + (r.bias ? (double)r.bias[e] : 0.0) : kNone;
            if (!(choice[v] > kNone))
                choice[v] = kNone;
        }
        if (r.topk_groups < r.groups) {
            const int per = r.experts / r.groups;
            double *value = choice_lds + r.experts;
#pragma unroll
            for (int v = 0; v < VPL; ++v)
                if (v * 64 + lane < r.experts)
                    choice_lds[v * 64 + lane] = choice[v];
            __syncthreads();
            for (int g = lane; g < r.groups; g += 64) {
                double first = kNone, second = kNone;
                for (int i = 0; i < per; ++i) {
                    const double cv = choice_lds[g * per + i];
                    if (cv > first) {
                        second = first;
                        first = cv;
                    } else if (cv > second) {
                        second = cv;
                    }
                }
                value[g] = r.group_top == 2 && second > kNone ? first + second : first;
            }
            __syncthreads();
            // chosen groups are marked by NaN
            for (int i = 0; i < r.topk_groups; ++i) {
                double best = kNone;
                int at = r.groups;
                for (int g = lane; g < r.groups; g += 64)
                    if (value[g] > best) {
                        best = value[g];
                        at = g;
                    }
                wave_argmax(best, at);
                if (!(best > kNone))
                    break;
                __syncthreads();
                if (lane == 0)
                    value[at] = __builtin_nan("");
                __syncthreads();
            }
#pragma unroll
            for (int v = 0; v < VPL; ++v) {
                const int e = v * 64 + lane;
                if (e < r.experts) {
                    const double gv = value[e / per];
                    if (gv == gv)
                        choice[v] = kNone;
                }
            }
            __syncthreads();
        }
        double my_score = 0.0, sum = 0.0;
        int my_index = -1;
        for (int j = 0; j < r.k; ++j) {
            double best = kNone;
            int at = r.experts;
#pragma unroll
            for (int v = 0; v < VPL; ++v)
                if (choice[v] > best) {
                    best = choice[v];
                    at = v * 64 + lane;
                }
            wave_argmax(best, at);
            if (!(best > kNone))
                break;
            double s = 0.0;
#pragma unroll
            for (int v = 0; v < VPL; ++v)
                if (at == v * 64 + lane) {
                    choice[v] = kNone;
                    s = score[v];
                }
            s = __shfl(s, at & 63);
            sum += s;
            if (lane == j) {
                my_index = at;
                my_score = s;
            }
        }
        if (lane < r.k) {
            double w = my_score;
            if (r.renormalise)
                w = sum > 0.0 ? w / sum : 0.0;
            r.index[t * r.k + lane] = my_index;
            r.weight[t * r.k + lane] = (float)(w * (double)r.scale);
        }
    }
}

template <class T>
hipError_t launch_route_typed(const RouteArgs &r, hipStream_t stream)
{
    const dim3 grid((unsigned)(r.tokens < 256 * 64 ? r.tokens : 256 * 64));
    const size_t lds = (size_t)(r.experts + r.groups) * sizeof(double);
    const int vpl = (r.experts + 63) / 64;
    if (vpl <= 1)
        hipLaunchKernelGGL((route_tokens<T, 1>), grid, dim3(64), lds, stream, r);
    else if (vpl <= 2)
        hipLaunchKernelGGL((route_tokens<T, 2>), grid, dim3(64), lds, stream, r);
    else if (vpl <= 4)
        hipLaunchKernelGGL((route_tokens<T, 4>), grid, dim3(64), lds, stream, r);
    else if (vpl <= 8)
        hipLaunchKernelGGL((route_tokens<T, 8>), grid, dim3(64), lds, stream, r);
    else
        hipLaunchKernelGGL((route_tokens<T, 16>), grid, dim3(64), lds, stream, r);
    return hipGetLastError();
}

// ---- the order of rows by expert: a stable counting sort ---------------------------------------
//
// The assignments are cut into nb chunks, one per workgroup (at most kMaxChunks, of kChunk assignments or
// more).  dispatch_count counts each chunk's experts; dispatch_scan turns each expert's counts into the
// number before each chunk; dispatch_place gives every assignment its slot: the slots of the experts before
// it, of its expert in the chunks before, in the waves before (each wave has a contiguous share of the chunk)
// and in its wave before it, the last by matching the lanes of equal expert bit by bit.  Every sum is of
// whole numbers and every position follows from the order alone, so the result is the same each time.
// Up to kChunk assignments take dispatch_place alone, in one workgroup.
constexpr int kThreads = 1024, kWaves = kThreads / 64;
constexpr int64_t kChunk = 4096, kMaxChunks = 1024;

int64_t chunk_of(int64_t n)
{
    const int64_t c = (n + kMaxChunks - 1) / kMaxChunks;
    return c <= kChunk ? kChunk : (c + kThreads - 1) / kThreads * kThreads;
}

// Exclusive scan over the workgroup; `total` gets the sum.  `sums`: kWaves + 1 ints of LDS.
__device__ __forceinline__ int block_scan(int v, int *sums, int &total)
{
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    int upto = v;
#pragma unroll
    for (int d = 1; d < 64; d <<= 1) {
        const int o = __shfl_up(upto, d);
        upto += lane >= d ? o : 0;
    }
    if (lane == 63)
        sums[wave] = upto;
    __syncthreads();
    int before = 0;
    total = 0;
#pragma unroll
    for (int w = 0; w < kWaves; ++w) {
        const int s = sums[w];
        before += w < wave ? s : 0;
        total += s;
    }
    __syncthreads();
    return before + upto - v;
}

__global__ __launch_bounds__(kThreads) void dispatch_count(DispatchArgs d, int64_t chunk, int nb)
{
    extern __shared__ int counts[];  // [experts]
    for (int e = threadIdx.x; e < d.experts; e += kThreads)
        counts[e] = 0;
    __syncthreads();
    const int64_t begin = blockIdx.x * chunk, end = begin + chunk < d.n ? begin + chunk : d.n;
    for (int64_t i = begin + threadIdx.x; i < end; i += kThreads) {
        const int e = d.index[i];
        if ((unsigned)e < (unsigned)d.experts)
            atomicAdd(&counts[e], 1);
    }
    __syncthreads();
    for (int e = threadIdx.x; e < d.experts; e += kThreads)
        d.workspace[(int64_t)e * nb + blockIdx.x] = counts[e];
}

__global__ __launch_bounds__(kThreads) void dispatch_scan(DispatchArgs d, int nb)
{
    __shared__ int sums[kWaves];
    int *row = d.workspace + (int64_t)blockIdx.x * nb;
    const int v = (int)threadIdx.x < nb ? row[threadIdx.x] : 0;
    int total;
    const int before = block_scan(v, sums, total);
    if ((int)threadIdx.x < nb)
        row[threadIdx.x] = before;
    if (threadIdx.x == 0)
        d.workspace[(int64_t)d.experts * nb + blockIdx.x] = total;
}

// ONE: the only workgroup, which counts for itself.
template <bool ONE>
__global__ __launch_bounds__(kThreads) void dispatch_place(DispatchArgs d, int64_t chunk, int nb)
{
    extern __shared__ int next[];  // [kWaves][experts]: counts, then the next slot
    __shared__ int sums[kWaves];
    const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6, E = d.experts;
    for (int i = tid; i < kWaves * E; i += kThreads)
        next[i] = 0;
    __syncthreads();
    const int64_t share = chunk / kWaves;
    const int64_t block0 = blockIdx.x * chunk, block1 = block0 + chunk < d.n ? block0 + chunk : d.n;
    const int64_t begin = block0 + wave * share, end = begin + share < block1 ? begin + share : block1;
    int *mine = next + wave * E;
    for (int64_t i = begin + lane; i < end; i += 64) {
        const int e = d.index[i];
        if ((unsigned)e < (unsigned)E)
            atomicAdd(&mine[e], 1);
    }
    __syncthreads();
    int count = 0;
    if (tid < E) {
        if constexpr (ONE)
            for (int w = 0; w < kWaves; ++w)
                count += next[w * E + tid];
        else
            count = d.workspace[(int64_t)E * nb + tid];
    }
    int total;
    const int base = block_scan(count, sums, total);
    if (tid < E) {
        int at = base + (ONE ? 0 : d.workspace[(int64_t)tid * nb + blockIdx.x]);
        for (int w = 0; w < kWaves; ++w) {
            const int in_wave = next[w * E + tid];
            next[w * E + tid] = at;
            at += in_wave;
        }
        if (blockIdx.x == 0) {
            d.offsets[tid] = base;
            if (tid == 0)
                d.offsets[E] = total;
        }
    }
    __syncthreads();
    int bits = 0;
    while ((1 << bits) < E)
        ++bits;
    for (int64_t i0 = begin; i0 < end; i0 += 64) {
        const int64_t i = i0 + lane;
        const int e = i < end ? d.index[i] : -1;
        const bool live = (unsigned)e < (unsigned)E;
        unsigned long long peers = __ballot(live);
        for (int b = 0; b < bits; ++b) {
            const unsigned long long set = __ballot((e >> b) & 1);
            peers &= (e >> b) & 1 ? set : ~set;
        }
        const int rank = __popcll(peers & ((1ull << lane) - 1));
        int slot = -1;
        if (live)
            slot = mine[e] + rank;
        __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");  // every lane has read before one adds
        __builtin_amdgcn_wave_barrier();
        if (live && rank == 0)
            mine[e] += __popcll(peers);
        __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
        __builtin_amdgcn_wave_barrier();
        if (i < end) {
            d.places[i] = slot;
            if (live)
                d.slots[slot] = (int)i;
        }
    }
    for (int64_t i = block0 + tid; i < block1; i += kThreads)  // slots not in use
        if (i >= total)
            d.slots[i] = -1;
}

}  // namespace

hipError_t launch_route(const RouteArgs &r, int dtype, hipStream_t stream)
{
    return dtype == kFp16 ? launch_route_typed<_Float16>(r, stream)
           : dtype == kBf16 ? launch_route_typed<__bf16>(r, stream)
                            : launch_route_typed<float>(r, stream);
}

int64_t dispatch_workspace_entries(int64_t n, int experts)
{
    const int64_t chunk = chunk_of(n), nb = (n + chunk - 1) / chunk;
    return nb <= 1 ? 0 : experts * (nb + 1);
}

hipError_t launch_dispatch(const DispatchArgs &d, hipStream_t stream)
{
    const int64_t chunk = chunk_of(d.n);
    const int nb = (int)((d.n + chunk - 1) / chunk);
    const size_t lds = (size_t)d.experts * sizeof(int);
    if (nb <= 1) {
        hipLaunchKernelGGL(dispatch_place<true>, dim3(1), dim3(kThreads), kWaves * lds, stream, d, chunk, 1);
        return hipGetLastError();
    }
    hipLaunchKernelGGL(dispatch_count, dim3(nb), dim3(kThreads), lds, stream, d, chunk, nb);
    hipError_t err = hipGetLastError();
    if (err == hipSuccess) {
        hipLaunchKernelGGL(dispatch_scan, dim3(d.experts), dim3(kThreads), 0, stream, d, nb);
        err = hipGetLastError();
    }
    if (err == hipSuccess) {
        hipLaunchKernelGGL(dispatch_place<false>, dim3(nb), dim3(kThreads), kWaves * lds, stream, d, chunk, nb);
        err = hipGetLastError();
    }
    return err;
}

}  // namespace mlpk
