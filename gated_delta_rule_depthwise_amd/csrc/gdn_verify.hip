// gdn_verify.hip -- drafted tokens against the target's probabilities, from given random
// numbers, on gfx950.
//
// Speculative sampling: draft t is accepted while u_t q_t(d_t) < p_t(d_t); with a drafts
// accepted, the next token is drawn from r = max(p_a - q_a, 0) (p_a when none was refused) by
// inverting its running sum at u_T * sum(r). The call reads one row of p, and one of q where
// a draft was refused, and is bound by HBM for a batch and by latency for one stream. A row
// is cut into parts that workgroups sum side by side (verify_sum_kernel, which finds a by
// itself from the 2 T probabilities concerned); verify_pick_kernel finds the part that holds
// the next token from those sums and looks through that part alone. Sums are held in float64, in
// a fixed order, so the token depends on nothing but the inputs.
#include <hip/hip_runtime.h>
#include <stdint.h>

#include "gdn_internal.h"

namespace gdn {

namespace {

typedef __bf16 bf16;

constexpr int THREADS = 256;

__device__ __forceinline__ float to_float(float x) { return x; }
__device__ __forceinline__ float to_float(bf16 x) { return (float)x; }

struct Row {
    int accepted;     // a
    int refused;      // 1: draft a was refused, its proposal's row applies
    int token;        // that draft
};

// The drafts accepted of stream b: all threads of the workgroup look at the tests side by
// side, the first that fails is the lowest set bit of some ballot.
template <typename T>
__device__ Row accept(const VerifyArgs &a, int b, int *first)
{
    int n = a.num_drafts ? a.num_drafts[b] : a.T;
    n = n < 0 ? 0 : n > a.T ? a.T : n;
    if (threadIdx.x == 0)
        *first = n;
    __syncthreads();
    for (int t = threadIdx.x; t < n; t += THREADS) {
        const int tok = a.tokens[(int64_t)b * a.T + t];
        bool ok = false;
        if (tok >= 0 && tok < a.V) {
            const double p = to_float(((const T *)a.target)[((int64_t)b * (a.T + 1) + t) * a.ld_target + tok]);
            const double q = a.draft ? to_float(((const T *)a.draft)[((int64_t)b * a.T + t) * a.ld_draft + tok]) : 1.f;
            ok = (double)a.u[(int64_t)b * (a.T + 1) + t] * q < p;  // exact: 24 + 24 bits
        }
        if (!ok)
            atomicMin(first, t);
    }
    __syncthreads();
    const int k = *first;
    return Row{k, k < n, k < n ? a.tokens[(int64_t)b * a.T + k] : -1};
}

// weights of element v: r = max(p - q, 0) and p; NaN and negative values count as zero
template <typename T> struct Weights {
    const T *p, *q;
    int one_hot;  // token whose proposal is 1 (draft == nullptr), or -1
    __device__ Weights(const VerifyArgs &a, int b, const Row &r)
    {
        p = (const T *)a.target + ((int64_t)b * (a.T + 1) + r.accepted) * a.ld_target;
        q = r.refused && a.draft ? (const T *)a.draft + ((int64_t)b * a.T + r.accepted) * a.ld_draft : nullptr;
        one_hot = r.refused && !a.draft ? r.token : -1;
    }
    __device__ float plain(int v) const { return fmaxf(to_float(p[v]), 0.f); }
    __device__ float rest(int v) const
    {
        const float x = to_float(p[v]) - (q ? to_float(q[v]) : v == one_hot ? 1.f : 0.f);
        return fmaxf(x, 0.f);
    }
};

// sum over the workgroup, in a fixed order; every thread gets it
__device__ double block_sum(double x, double *red)
{
#pragma unroll
    for (int m = 1; m < 64; m <<= 1)
        x += __shfl_xor(x, m);
    __syncthreads();
    if ((threadIdx.x & 63) == 0)
        red[threadIdx.x >> 6] = x;
    __syncthreads();
    x = 0.;
    for (int i = 0; i < THREADS / 64; ++i)
        x += red[i];
    return x;
}

template <typename T>
__global__ void __launch_bounds__(THREADS) verify_sum_kernel(const VerifyArgs a)
{
    __shared__ int first;
    __shared__ double red[THREADS / 64];
    const int b = blockIdx.x / a.nseg, sg = blockIdx.x % a.nseg;
    const Row row = accept<T>(a, b, &first);
    const Weights<T> w(a, b, row);
    const int v0 = sg * a.seg, v1 = a.V - v0 < a.seg ? a.V : v0 + a.seg;
    double r = 0., p = 0.;
    for (int v = v0 + threadIdx.x; v < v1; v += THREADS) {
        p += w.plain(v);
        r += w.rest(v);
    }
    r = block_sum(r, red);
    p = block_sum(p, red);
    if (threadIdx.x == 0) {
        double *out = a.part + ((int64_t)b * a.nseg + sg) * 2;
        out[0] = r, out[1] = p;
    }
}

template <typename T>
__global__ void __launch_bounds__(THREADS) verify_pick_kernel(const VerifyArgs a)
{
    __shared__ int first;
    __shared__ double cum[THREADS];
    __shared__ int found, last;
    const int b = blockIdx.x, tid = threadIdx.x;
    const Row row = accept<T>(a, b, &first);
    const Weights<T> w(a, b, row);
    const double *part = a.part + (int64_t)b * a.nseg * 2;
    // the part that holds the token: the first whose running sum passes the aim, or where
    // rounding leaves none the last that holds any weight
    double total = 0.;
    for (int i = 0; i < a.nseg; ++i)
        total += part[2 * i];
    const bool use_p = !(total > 0.);
    if (use_p) {
        total = 0.;
        for (int i = 0; i < a.nseg; ++i)
            total += part[2 * i + 1];
    }
    const double aim = (double)a.u[(int64_t)b * (a.T + 1) + a.T] * total;
    double before = 0.;
    int sg = -1;
    {
        double run = 0.;
        for (int i = 0; i < a.nseg; ++i) {
            const double x = part[2 * i + use_p];
            if (x > 0.)
                sg = i, before = run;
            run += x;
            if (run > aim)
                break;
        }
    }
    if (tid == 0)
        found = 0x7fffffff, last = -1;
    __syncthreads();
    if (sg >= 0) {
        // each thread a run of consecutive elements of the part
        const int v0 = sg * a.seg, v1 = a.V - v0 < a.seg ? a.V : v0 + a.seg;
        const int per = (v1 - v0 + THREADS - 1) / THREADS;
        const int64_t e0 = (int64_t)v0 + (int64_t)tid * per;
        const int lo = e0 < v1 ? (int)e0 : v1, hi = v1 - lo < per ? v1 : lo + per;
        double sum = 0.;
        int mine = -1;
        for (int v = lo; v < hi; ++v) {
            const float x = use_p ? w.plain(v) : w.rest(v);
            sum += x;
            if (x > 0.f)
                mine = v;
        }
        cum[tid] = sum;
        if (mine >= 0)
            atomicMax(&last, mine);
        __syncthreads();
        double run = before;
        for (int i = 0; i < tid; ++i)
            run += cum[i];
        if (run <= aim) {
            for (int v = lo; v < hi; ++v) {
                run += use_p ? w.plain(v) : w.rest(v);
                if (run > aim) {
                    atomicMin(&found, v);
                    break;
                }
            }
        } else if (tid > 0) {
            // an earlier thread's run has it
        }
        __syncthreads();
    }
    if (tid == 0) {
        a.accepted[b] = row.accepted;
        a.next[b] = found != 0x7fffffff ? found : last;
        if (a.len)
            a.len[b] += row.accepted + 1;
    }
}

template <typename T> hipError_t verify_t(const VerifyArgs &a, hipStream_t s)
{
    hipLaunchKernelGGL((verify_sum_kernel<T>), dim3((unsigned)(a.B * a.nseg)), dim3(THREADS), 0, s, a);
    if (hipError_t e = hipGetLastError(); e != hipSuccess)
        return e;
    hipLaunchKernelGGL((verify_pick_kernel<T>), dim3((unsigned)a.B), dim3(THREADS), 0, s, a);
    return hipGetLastError();
}

}  // namespace

hipError_t launch_verify(int dtype, const VerifyArgs &a, hipStream_t s)
{
    return dtype ? verify_t<bf16>(a, s) : verify_t<float>(a, s);
}

}  // namespace gdn
