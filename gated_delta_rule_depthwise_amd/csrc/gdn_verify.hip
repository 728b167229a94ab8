// gdn_verify.hip -- drafted tokens against the target's probabilities, from given random
// numbers, on gfx950.
//
// Speculative sampling: draft t is accepted while u_t q_t(d_t) < p_t(d_t); with a drafts
// accepted, the next token is drawn from r = max(p_a - q_a, 0) (p_a when none was refused) by
// inverting its running sum at u_T * sum(r). The call reads one row of p, and one of q where
// a draft was refused: a batch is bound by HBM, one stream by latency. One workgroup of 16
// waves per stream sums the row, a stretch per wave, and narrows down to at most 8192 elements
// (which come from L2 then), 8 per thread, whose running sum gives the token. Where a few
// streams have long rows (launch_verify), workgroups sum parts of the rows side by side first
// (verify_sum_kernel). Sums are held in float64 and taken in a fixed order, so the token
// depends on nothing but the inputs. Measured: 256 streams of 131072 bf16 weights 27 us (a
// workgroup per CU, so the tests before a row and the search after it are not hidden; the rows
// alone take about 20 us at 5.2 TB/s), one stream of 32000 weights 9.5 us (four round trips
// to memory in a chain: drafts, their probabilities, the row, the stretch again).
#include <hip/hip_runtime.h>
#include <stdint.h>

#include "gdn_draft.h"

namespace gdn {

namespace {

typedef __bf16 bf16;

constexpr int PICK_THREADS = 1024, PICK_WAVES = PICK_THREADS / 64;
constexpr int SUM_THREADS = 256;
constexpr int VE = 8;              // adjacent elements per lane and step
constexpr int STEP = 64 * VE;      // elements per wave and step
constexpr int LAST = PICK_THREADS * VE;  // elements looked at one by one

__device__ __forceinline__ float to_float(float x) { return x; }
__device__ __forceinline__ float to_float(bf16 x) { return (float)x; }

// 8 adjacent elements from any element address: rows need no more alignment than that, and
// the hardware takes 16-byte loads at any address
typedef uint32_t u32x4_any __attribute__((ext_vector_type(4), aligned(2)));
typedef float f32x4_any __attribute__((ext_vector_type(4), aligned(4)));

typedef float Eight __attribute__((ext_vector_type(VE)));

__device__ __forceinline__ Eight load8(const bf16 *p)
{
    const u32x4_any u = *(const u32x4_any *)p;
    Eight r;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        r[2 * i] = __uint_as_float(u[i] << 16);
        r[2 * i + 1] = __uint_as_float(u[i] & 0xffff0000u);
    }
    return r;
}

__device__ __forceinline__ Eight load8(const float *p)
{
    const f32x4_any a = *(const f32x4_any *)p, b = *(const f32x4_any *)(p + 4);
    return Eight{a[0], a[1], a[2], a[3], b[0], b[1], b[2], b[3]};
}

template <typename T> __device__ __forceinline__ Eight load8(const T *p, int n)
{
    Eight r = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
    if (n >= VE) {
        r = load8(p);
    } else {
#pragma unroll
        for (int i = 0; i < VE; ++i)
            if (i < n)
                r[i] = to_float(p[i]);
    }
    return r;
}

// The drafts accepted of stream b, and the number of its drafts: the workgroup's threads look
// at the tests side by side; the first that fails counts.
template <typename T, int THREADS>
__device__ __forceinline__ int accept(const VerifyArgs &a, int b, int *first, int &n)
{
    n = a.num_drafts ? a.num_drafts[b] : a.T;
    if (threadIdx.x == 0)
        *first = a.T;
    __syncthreads();
    for (int t = threadIdx.x; t < a.T; t += THREADS) {
        const int tok = a.tokens[(int64_t)b * a.T + t];
        const float u = a.u[(int64_t)b * (a.T + 1) + t];
        bool ok = false;
        if (tok >= 0 && tok < a.V) {
            const double p = to_float(((const T *)a.target)[((int64_t)b * (a.T + 1) + t) * a.ld_target + tok]);
            const double q = a.draft ? to_float(((const T *)a.draft)[((int64_t)b * a.T + t) * a.ld_draft + tok]) : 1.f;
            ok = (double)u * q < p;  // the product is exact: 24 + 24 bits
        }
        if (!ok)
            atomicMin(first, t);
    }
    n = n < 0 ? 0 : n > a.T ? a.T : n;
    __syncthreads();
    return *first < n ? *first : n;
}

// The weights r = max(p - q, 0) of a stream's next token; NaN and negative values count as
// zero. q: the refused draft's proposal (nullptr: none, or 1 at token one_hot alone).
template <typename T> struct Weights {
    const T *p, *q;
    int one_hot;
    __device__ Weights(const VerifyArgs &a, int b, int accepted, int n)
    {
        const bool refused = accepted < n;
        p = (const T *)a.target + ((int64_t)b * (a.T + 1) + accepted) * a.ld_target;
        q = refused && a.draft ? (const T *)a.draft + ((int64_t)b * a.T + accepted) * a.ld_draft : nullptr;
        one_hot = refused && !a.draft ? a.tokens[(int64_t)b * a.T + accepted] : -1;
    }
    __device__ __forceinline__ Eight combine(int v, Eight x, Eight y) const
    {
#pragma unroll
        for (int i = 0; i < VE; ++i) {
            const float s = q ? y[i] : v + i == one_hot ? 1.f : 0.f;
            x[i] = fmaxf(x[i] - s, 0.f);
        }
        return x;
    }
    // elements v .. v+7, those at or past `hi` as 0
    __device__ __forceinline__ Eight at(int v, int hi) const
    {
        const int n = hi - v;
        const Eight x = load8(p + v, n);
        Eight y = x;
        if (q)
            y = load8(q + v, n);
        return combine(v, x, y);
    }
};

__device__ __forceinline__ double sum8(Eight e)
{
    double s = 0.;
#pragma unroll
    for (int i = 0; i < VE; ++i)
        s += e[i];
    return s;
}

// Sum of the weights of elements lo .. hi-1 over a wave; every lane gets it. Four steps'
// loads are in flight together; the lane that holds the row's end has its own.
template <typename T> __device__ __forceinline__ double wave_sum(const Weights<T> w, int lo, int hi)
{
    const int lane = threadIdx.x & 63;
    double sum = 0.;
    int v = lo + lane * VE;
    for (int full = (hi - lo) / (4 * STEP); full > 0; --full, v += 4 * STEP) {
        Eight x[4], y[4];
#pragma unroll
        for (int i = 0; i < 4; ++i)
            x[i] = load8(w.p + v + i * STEP);
        if (w.q) {
#pragma unroll
            for (int i = 0; i < 4; ++i)
                y[i] = load8(w.q + v + i * STEP);
        }
#pragma unroll
        for (int i = 0; i < 4; ++i)
            sum += sum8(w.combine(v + i * STEP, x[i], y[i]));
    }
    if (hi - v >= VE) {
        Eight x[4], y[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            x[i] = y[i] = Eight{0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
            if (hi - v >= i * STEP + VE) {
                x[i] = load8(w.p + v + i * STEP);
                if (w.q)
                    y[i] = load8(w.q + v + i * STEP);
            }
        }
#pragma unroll
        for (int i = 0; i < 4; ++i)
            if (hi - v >= i * STEP + VE)
                sum += sum8(w.combine(v + i * STEP, x[i], y[i]));
    }
    const int end = hi - (hi - lo) % VE;  // the elements left over, fewer than a load's
    if (end < hi && lane == 0)
        sum += sum8(w.at(end, hi));
#pragma unroll
    for (int m = 1; m < 64; m <<= 1)
        sum += __shfl_xor(sum, m);
    return sum;
}

template <typename T>
__global__ void __launch_bounds__(SUM_THREADS) verify_sum_kernel(const VerifyArgs a)
{
    constexpr int WAVES = SUM_THREADS / 64;
    __shared__ int first;
    __shared__ double red[WAVES];
    const int b = blockIdx.x / a.nseg, sg = blockIdx.x % a.nseg, wave = threadIdx.x >> 6;
    int n;
    const int acc = accept<T, SUM_THREADS>(a, b, &first, n);
    const Weights<T> w(a, b, acc, n);
    // a part is a multiple of 4 * STEP elements, but for the row's end
    const int v0 = sg * a.seg, v1 = a.V - v0 < a.seg ? a.V : v0 + a.seg;
    const int per = a.seg / WAVES, lo = v0 + wave * per;
    const int hi = lo >= v1 ? lo : v1 - lo < per ? v1 : lo + per;
    const double sum = wave_sum(w, lo, hi);
    if ((threadIdx.x & 63) == 0)
        red[wave] = sum;
    __syncthreads();
    if (threadIdx.x == 0) {
        double s = 0.;
        for (int i = 0; i < WAVES; ++i)
            s += red[i];
        a.part[(int64_t)b * a.nseg + sg] = s;
        if (sg == 0) {
            a.info[2 * b] = acc;
            a.info[2 * b + 1] = n;
        }
    }
}

// Running sum of n <= 64 values, lane i those of 0 .. i (lanes past n: all of them)
__device__ __forceinline__ double scan(const double *sums, int n, double &own)
{
    const int lane = threadIdx.x & 63;
    own = lane < n ? sums[lane] : 0.;
    double run = own;
#pragma unroll
    for (int m = 1; m < 64; m <<= 1) {
        const double y = __shfl_up(run, m);
        run += lane >= m ? y : 0.;
    }
    return run;
}

template <typename T, bool PARTS>
__global__ void __launch_bounds__(PICK_THREADS) verify_pick_kernel(const VerifyArgs a)
{
    __shared__ int first, hit, last;
    __shared__ double sums[64];
    const int b = blockIdx.x, tid = threadIdx.x, lane = tid & 63;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const float u = a.u[(int64_t)b * (a.T + 1) + a.T];
    int acc, n, nsum = PICK_WAVES;
    if (tid == 0)
        hit = 0x7fffffff, last = -1;
    if constexpr (PARTS)
        acc = a.info[2 * b], n = a.info[2 * b + 1];
    else
        acc = accept<T, PICK_THREADS>(a, b, &first, n);
    Weights<T> w(a, b, acc, n);

    int lo = 0, hi = a.V, per = 0;
    // sums of 16 stretches of `per` elements of lo .. hi-1
    const auto cut = [&]() {
        per = (hi - lo + PICK_WAVES - 1) / PICK_WAVES;
        per = (per + VE - 1) / VE * VE;
        const int64_t at = (int64_t)lo + (int64_t)wave * per;
        const int l = at < hi ? (int)at : hi, h = hi - l < per ? hi : l + per;
        const double s = wave_sum(w, l, h);
        __syncthreads();
        if (lane == 0)
            sums[wave] = s;
        __syncthreads();
        nsum = PICK_WAVES;
    };
    // the same of 8 elements per thread: x, their sum `own`, and its running sum in the wave
    Eight x;
    double own, run;
    const auto load_all = [&]() {
        x = w.at(lo + tid * VE < hi ? lo + tid * VE : hi, hi);
        own = sum8(x);
        run = own;
#pragma unroll
        for (int m = 1; m < 64; m <<= 1) {
            const double y = __shfl_up(run, m);
            run += lane >= m ? y : 0.;
        }
        __syncthreads();
        if (lane == 63)
            sums[wave] = run;
        __syncthreads();
        nsum = PICK_WAVES;
    };
    double part, upto, all, before = 0.;  // lane i: sum i, and those of 0 .. i
    bool loaded = false;
    for (int pass = 0; pass < 2; ++pass) {
        if (hi <= LAST)
            load_all(), loaded = true;
        else if (PARTS && pass == 0) {
            if (tid < a.nseg)
                sums[tid] = a.part[(int64_t)b * a.nseg + tid];
            nsum = a.nseg, per = a.seg;
            __syncthreads();
        } else
            cut();
        upto = scan(sums, nsum, part), all = __shfl(upto, 63);
        if (all > 0. || (!w.q && w.one_hot < 0))
            break;
        w.q = nullptr, w.one_hot = -1;  // nothing is left over: draw from p itself
    }
    const double aim = (double)u * all;
    while (hi - lo > LAST) {
        // the first stretch at which the running sum passes the aim, or where rounding leaves
        // none the last that is not zero
        const uint64_t pass = __ballot(part > 0. && before + upto > aim), any = __ballot(part > 0.);
        const int at = pass ? __builtin_ctzll(pass) : any ? 63 - __builtin_clzll(any) : 0;
        before += __shfl(upto, at) - __shfl(part, at);
        lo = lo + at * per;
        hi = hi - lo < per ? hi : lo + per;
        if (hi - lo <= LAST)
            break;
        cut();
        upto = scan(sums, nsum, part);
    }
    if (!loaded) {
        load_all();
        upto = scan(sums, nsum, part);
    }
    // element by element: the first weight at which the running sum passes the aim, or the last
    before += __shfl(upto, wave) - __shfl(part, wave) + (run - own);
    int my_hit = -1, my_last = -1;
#pragma unroll
    for (int i = 0; i < VE; ++i) {
        before += x[i];
        if (x[i] > 0.f) {
            my_last = i;
            if (my_hit < 0 && before > aim)
                my_hit = i;
        }
    }
    const uint64_t hits = __ballot(my_hit >= 0), any = __ballot(my_last >= 0);
    if (hits && lane == __builtin_ctzll(hits))
        atomicMin(&hit, lo + tid * VE + my_hit);
    if (any && lane == 63 - __builtin_clzll(any))
        atomicMax(&last, lo + tid * VE + my_last);
    __syncthreads();
    if (tid == 0) {
        a.accepted[b] = acc;
        a.next[b] = hit != 0x7fffffff ? hit : last;
        if (a.len)
            a.len[b] += acc + 1;
    }
}

template <typename T> hipError_t verify_t(const VerifyArgs &a, hipStream_t s)
{
    // One workgroup per row where rows are short or fill the device; a few long rows by parts
    // and a second launch (1 stream of 131072: 10.3 us against 16.0 us, 96 streams of 200000:
    // 28.3 us against 41.0 us; 1 stream of 32000: 9.8 us against 9.4 us, 256 streams of 131072:
    // 47.0 us against 43.4 us).
    if (a.V <= 32768 || a.B >= 128) {
        hipLaunchKernelGGL((verify_pick_kernel<T, false>), dim3((unsigned)a.B), dim3(PICK_THREADS), 0, s, a);
        return hipGetLastError();
    }
    hipLaunchKernelGGL((verify_sum_kernel<T>), dim3((unsigned)(a.B * a.nseg)), dim3(SUM_THREADS), 0, s, a);
    if (hipError_t e = hipGetLastError(); e != hipSuccess)
        return e;
    hipLaunchKernelGGL((verify_pick_kernel<T, true>), dim3((unsigned)a.B), dim3(PICK_THREADS), 0, s, a);
    return hipGetLastError();
}

}  // namespace

hipError_t launch_verify(int dtype, const VerifyArgs &a, hipStream_t s)
{
    return dtype ? verify_t<bf16>(a, s) : verify_t<float>(a, s);
}

}  // namespace gdn
