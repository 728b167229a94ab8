// gdn_draft.hip -- drafted tokens on gfx950: T tokens per stream against states that are only
// read (draft_kernel), and the streams' tapes worked into their states (fold_kernel).
//
// With h the state in memory, k_j, d_j the entries of a stream's tape (or its new tokens)
// and G the running sum of log-gates from h on, the new token t gives
//   y_t = h^T (e^{G_t} k_t) + sum_{j before t} (k_j . e^{G_t - G_j} k_t) d_j,
//   d_t = beta_t (v_t - y_t),
//   o_t = h^T (e^{G_t} q_t) + sum_{j up to t} (k_j . e^{G_t - G_j} q_t) d_j,
// so the state is read once for all the tokens (and streams) of a workgroup and never
// written: with short tapes the call moves about half the bytes of an in-place decode step.
// The products with h and with the tape's keys run on fp32 MFMA (a workgroup's 256 products
// of 16 x 16 x 4 with a 128 x 128 state take 2048 cycles of each SIMD, its 64 KiB about 7000
// cycles of the CU's share of HBM; operands of fewer bits would need three products each for
// fp32's precision); the tape's updates are added per column on the VALU, where a stream's
// rows can be kept apart, and the part among the new tokens is a triangular solve of at most
// 16 steps per column. HBM bounds the large calls (256 streams x 8 tokens x 32 heads of 128 x
// 128: 169 us, 842 MB, 5.0 TB/s, where a device copy reaches 5.2); between those and the small
// ones a workgroup's chain of waits does (rows, L2, scores, products, solve: about 30 000
// cycles, four workgroups per CU; 64 streams x 5 tokens: 45 us, 4.3 TB/s), and the smallest
// take one such chain (1 stream x 1 token: 8.7 us).
//
// fold: h_out = diag(e^{G_n}) h + sum_j diag(e^{G_n - G_j}) k_j d_j^T, a rank-n update on
// fp32 MFMA of a state that is read and written once: bound by HBM (64 streams x 32 heads,
// tapes of 1 to 16: 57 us, 300 MB, 5.2 TB/s).
#include <hip/hip_runtime.h>
#include <stdint.h>

#include "gdn.h"
#include "gdn_draft.h"

namespace gdn {

namespace {

typedef __bf16 bf16;
typedef float f32x4 __attribute__((ext_vector_type(4)));

constexpr int THREADS = 256;
constexpr int WAVES = THREADS / 64;

__device__ __forceinline__ f32x4 load_nt4(const float *p)
{
    return __builtin_nontemporal_load((const f32x4 *)p);
}
__device__ __forceinline__ f32x4 load4(const float *p) { return *(const f32x4 *)p; }
__device__ __forceinline__ f32x4 load4(const bf16 *p)
{
    const uint2 u = *(const uint2 *)p;
    return f32x4{__uint_as_float(u.x << 16), __uint_as_float(u.x & 0xffff0000u),
                 __uint_as_float(u.y << 16), __uint_as_float(u.y & 0xffff0000u)};
}

__device__ __forceinline__ f32x4 zero4() { return f32x4{0.f, 0.f, 0.f, 0.f}; }

__device__ __forceinline__ f32x4 mfma4(float a, float b, f32x4 c)
{
    return __builtin_amdgcn_mfma_f32_16x16x4f32(a, b, c, 0, 0, 0);
}

// two adjacent channels of a raw row, kept as loaded (the tape takes the same bits)
template <typename T> struct Pair;
template <> struct Pair<bf16> {
    typedef uint32_t raw;
    static __device__ __forceinline__ float lo(raw r) { return __uint_as_float(r << 16); }
    static __device__ __forceinline__ float hi(raw r) { return __uint_as_float(r & 0xffff0000u); }
    static __device__ __forceinline__ raw make(const bf16 *a, const bf16 *b)
    {
        return (uint32_t)*(const uint16_t *)a | (uint32_t)*(const uint16_t *)b << 16;
    }
};
template <> struct Pair<float> {
    typedef float2 raw;
    static __device__ __forceinline__ float lo(raw r) { return r.x; }
    static __device__ __forceinline__ float hi(raw r) { return r.y; }
    static __device__ __forceinline__ raw make(const float *a, const float *b)
    {
        return float2{*a, *b};
    }
};

__device__ __forceinline__ float silu(float x)
{
    return x * __builtin_amdgcn_rcpf(1.f + __expf(-x));
}

// Cross-lane moves within a row of 16 lanes (DPP: an operand modifier, no LDS round trip). A
// lane whose source lies outside its row gets 0.
template <int CTRL> __device__ __forceinline__ float dpp(float x)
{
    return __builtin_bit_cast(
        float, __builtin_amdgcn_update_dpp(0, __builtin_bit_cast(int, x), CTRL, 0xf, 0xf, true));
}
constexpr int DPP_SHR = 0x110;  // + n: from the lane n below

// Sum over a row of 16 lanes; every lane gets it.
__device__ __forceinline__ float row_sum(float x)
{
    x += dpp<0xb1>(x);   // quad_perm 1,0,3,2
    x += dpp<0x4e>(x);   // quad_perm 2,3,0,1
    x += dpp<0x141>(x);  // mirrored half row
    x += dpp<0x140>(x);  // mirrored row
    return x;
}

// Sum over the lanes 0 .. l of a row, at lane l.
__device__ __forceinline__ float row_scan(float x)
{
    x += dpp<DPP_SHR + 1>(x);
    x += dpp<DPP_SHR + 2>(x);
    x += dpp<DPP_SHR + 4>(x);
    x += dpp<DPP_SHR + 8>(x);
    return x;
}

// Sum over groups of N lanes (16, 32 or 64), every lane gets it.
template <int N> __device__ __forceinline__ float group_sum(float x)
{
    x = row_sum(x);
#pragma unroll
    for (int m = 16; m < N; m <<= 1)
        x += __shfl_xor(x, m);
    return x;
}

// One workgroup: one state (prefix, head) and a tile of up to TOK tokens of its streams, ns
// streams of T tokens. Rows of the products are the tokens' keys (rows 0 .. TOK-1) and
// queries (TOK .. 2*TOK-1).
template <int DK, int DV, bool KDA, int TOK> struct DraftShape {
    static constexpr int R = 2 * TOK;          // rows of the products
    static constexpr int MT = R / 16;          // 16-row MFMA tiles
    static constexpr int NS = 8;               // streams per tile, at most
    static constexpr int CG = DV / 64;         // 64-column groups, one wave (or more) each
    static constexpr int RS = WAVES / CG;      // waves that share a column group's rows
    static constexpr int RW = DK / RS;         // rows of h per wave
    static constexpr int LDK = DK + 4;         // row stride of the key tile
    static constexpr int LDS_ = 20;            // row stride of the score tiles
    static constexpr int G = THREADS / DV;     // threads per column
    static constexpr int EG = 16 / G;          // entries of a tape block per thread of a column
    static constexpr int GW = KDA ? DK : 1;    // log-gates per token
    static constexpr int CQ = DK / WAVES / 16; // 16-channel groups per wave in the scores
    static_assert(G == RS, "a part of Y per thread of a column");
    // LDS, in floats; the partial products Y overlay what is dead by then
    static constexpr int KQ = 0;
    static constexpr int Y = KQ + R * LDK;
    static constexpr int SP = Y;                              // a round's scores, by wave
    static constexpr int FS = SP + 2 * WAVES * R * LDS_;      // and their sums
    static constexpr int GK = FS + 2 * R * LDS_;              // KDA: new tokens' log-gates
    static constexpr int END1 = GK + (KDA ? TOK * DK : 0);
    static constexpr int END2 = Y + RS * R * DV;
    static constexpr int RUN = END1 > END2 ? END1 : END2;     // log-decay over a tape's newer blocks
    static constexpr int VD = RUN + NS * GW;                  // v
    static constexpr int CO = VD + TOK * DV;                  // coefficients among new tokens
    static constexpr int SM = CO + R * TOK;                   // small: see the kernel
    static constexpr int TOTAL = SM + 2 * TOK + NS + 32;
    static_assert(RW % 16 == 0 && DK % 16 == 0, "tile map");
    static_assert(TOTAL * 4 <= 80 * 1024, "LDS of two workgroups per CU (160 KiB)");
};

// Waves per SIMD the registers are held to: four workgroups of a CU hide each other's waits
// (256 streams x 8 tokens: 169 us with 4, 183 us with 3; channel gates, 32 x 4 tokens: 29.4 us
// with 4 and 18 registers spilled, 32.3 us with 3). Twice the tokens take the LDS of two.
template <int DK, int DV, bool KDA, int TOK> constexpr int draft_waves()
{
    return TOK == 16 ? 2 : DV <= 128 ? 4 : 3;
}

template <typename T, int DK, int DV, bool KDA, int K, int TOK>
__global__ void __launch_bounds__(THREADS, (draft_waves<DK, DV, KDA, TOK>())) draft_kernel(const DraftArgs a, int ntile)
{
    using S = DraftShape<DK, DV, KDA, TOK>;
    using P = Pair<T>;
    constexpr int W = K > 0 ? K - 1 : 0;
    constexpr int R = S::R, MT = S::MT, NS = S::NS, LDK = S::LDK, EG = S::EG, GW = S::GW;
    __shared__ __align__(16) float sm[S::TOTAL];
    float *const kq = sm + S::KQ, *const sp = sm + S::SP, *const fs = sm + S::FS;
    float *const gk = sm + S::GK, *const y = sm + S::Y, *const run = sm + S::RUN;
    float *const vd = sm + S::VD, *const co = sm + S::CO;
    float *const gam = sm + S::SM;        // [TOK] log-gates through each new token (GDN)
    float *const bet = gam + TOK;         // [TOK]
    int *const slen = (int *)(bet + TOK); // [NS] tape lengths, -1: stream left out
    float *const suf = (float *)(slen + NS);  // [2][16] log-decay after a block's entries (GDN)

    const int H = a.H, Hqk = a.Hqk, Tn = a.T, cap = a.tape.cap;
    // the tiles of one state run on one XCD (workgroups go to the 8 XCDs in turn), whose L2
    // then serves all but the first of them
    const int tile = (blockIdx.x >> 3) % ntile, ph = (blockIdx.x >> 3) / ntile * 8 + (blockIdx.x & 7);
    if (ph >= (a.B / a.share) * H)
        return;
    const int head = ph % H, pfx = ph / H;
    const int rep = H / Hqk, hq = head / rep;
    const bool own_qk = head % rep == 0;  // this workgroup writes the q/k head's tape entries
    const int nsmax = TOK / Tn < NS ? TOK / Tn : NS;
    const int s0 = tile * nsmax;
    const int ns = a.share - s0 < nsmax ? a.share - s0 : nsmax;
    const int b0 = pfx * a.share + s0, nt = ns * Tn;
    const int64_t row0 = (int64_t)b0 * Tn;
    const int64_t cd = 2 * (int64_t)Hqk * DK + (int64_t)H * DV;
    const int tid = threadIdx.x, lane = tid & 63;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int c16 = lane & 15, g4 = lane >> 4;
    const int cg = wave % S::CG, rs = wave / S::CG;
    const int col = tid % DV, grp = tid / DV;
    // stream of a token of the tile: exact for tok < 16, T <= 16 (the rounding of 256/T up
    // adds less than 16/256, which is below 1/T)
    const int inv_t = (256 + Tn - 1) / Tn;
    const auto stream_of = [&](int tok) { return tok * inv_t >> 8; };

    // tape lengths, -1 where a stream is left out: lane s of every wave has that of stream s,
    // its number of blocks (16 entries, newest first) and those of the streams before it
    int len_s = -1;
    if (lane < ns) {
        len_s = a.tape.len[b0 + lane];
        len_s = len_s < 0 || len_s > cap - Tn ? -1 : len_s;
    }
    if (tid < NS) {
        slen[tid] = len_s;
        if (tid < ns && len_s < 0 && a.tape.status && head == 0)
            atomicOr(a.tape.status, GDN_BAD_TAPE);
    }
    const auto tape_len = [&](int s) { return __builtin_amdgcn_readlane(len_s, s); };
    const int nb_s = (len_s + 15) >> 4;
    int upto = nb_s;
    upto += __builtin_amdgcn_update_dpp(0, upto, DPP_SHR + 1, 0xf, 0xf, true);
    upto += __builtin_amdgcn_update_dpp(0, upto, DPP_SHR + 2, 0xf, 0xf, true);
    upto += __builtin_amdgcn_update_dpp(0, upto, DPP_SHR + 4, 0xf, 0xf, true);
    const int nblk = __builtin_amdgcn_readlane(upto, NS - 1);
    // block blk < nblk of the tile's streams: its stream, and one past its newest entry
    const auto block_at = [&](int blk, int &s, int &hi) {
        s = __builtin_ctzll(__ballot(lane < NS && blk < upto));
        hi = tape_len(s) - 16 * (blk - __builtin_amdgcn_readlane(upto - nb_s, s));
    };

    // ---- loads of the front end: a thread takes two adjacent channels of every token --------
    constexpr int CP = (2 * DK + DV) / 2;
    static_assert(CP <= THREADS, "front end map");
    const int fc = 2 * tid, sec = fc < DK ? 0 : fc < 2 * DK ? 1 : 2;
    const int fe = sec == 0 ? fc : sec == 1 ? fc - DK : fc - 2 * DK;
    const int64_t fcol = sec == 2 ? (int64_t)head * DV + fe : (int64_t)hq * DK + fe;
    const int64_t ch = (sec == 0 ? 0 : (int64_t)sec * Hqk * DK) + fcol;
    typename P::raw raw[TOK], old[TOK][W > 0 ? W : 1];  // old: the window at a stream's first token
    float2 w[K > 0 ? K : 1];
    if (tid < CP) {
        const T *src = (const T *)(sec == 0 ? a.q : sec == 1 ? a.k : a.v) + row0 * a.ld + fcol;
#pragma unroll
        for (int tok = 0; tok < TOK; ++tok) {
            raw[tok] = typename P::raw{};
            if (tok < nt)
                raw[tok] = *(const typename P::raw *)(src + tok * a.ld);
        }
        if constexpr (K > 0) {
#pragma unroll
            for (int i = 0; i < K; ++i)
                w[i] = float2{a.conv_w[ch * K + i], a.conv_w[(ch + 1) * K + i]};
            const T *win = (const T *)a.conv_state_ptrs[pfx] + ch * W;
            const T *tr = (const T *)a.tape.raw + (int64_t)b0 * cap * cd + ch;
            const auto load_window = [&](int s, typename P::raw (&o)[W]) {
                const int n = tape_len(s);
                if (n >= W) {  // all on the tape
#pragma unroll
                    for (int i = 0; i < W; ++i)
                        o[i] = *(const typename P::raw *)(tr + ((int64_t)s * cap + n - W + i) * cd);
                } else {
#pragma unroll
                    for (int i = 0; i < W; ++i) {
                        const int m = n - W + i;
                        const bool tape = m >= 0;
                        const T *x = tape ? tr + ((int64_t)s * cap + m) * cd : win + (n < 0 ? i : W + m);
                        o[i] = P::make(x, x + (tape ? 1 : W));
                    }
                }
            };
            load_window(0, old[0]);
            if (ns > 1) {
                int s = 1, t = 1;
#pragma unroll
                for (int tok = 1; tok < TOK; ++tok) {
                    if (t == Tn) {
                        if (s < ns)
                            load_window(s, old[tok]);
                        t = 0, ++s;
                    }
                    ++t;
                }
            }
        }
    }
    // log-gates and betas of the new tokens
    float bet_r = 0.f, g_r = 0.f;
    if (tid >= THREADS - TOK && tid < THREADS - TOK + nt) {
        const int tok = tid - (THREADS - TOK);
        bet_r = a.beta[(row0 + tok) * H + head];
        if constexpr (!KDA)
            g_r = a.g[(row0 + tok) * H + head];
    }
    constexpr int GL = KDA ? (TOK * DK / 4 + THREADS - 1) / THREADS : 1;
    f32x4 g4r[GL];
    if constexpr (KDA) {
#pragma unroll
        for (int p = 0; p < GL; ++p) {
            const int i = tid + p * THREADS, tok = i / (DK / 4), c = 4 * (i % (DK / 4));
            g4r[p] = tok < nt ? load4(a.g + ((row0 + tok) * H + head) * DK + c) : zero4();
        }
    }

    // ---- loads of the first two tape blocks: a wave takes the keys' channels wave*DK/4 on (and
    // their log-gates), a thread some entries of its column's updates ------------------------
    constexpr int CQ = S::CQ;
    const int wc = wave * (DK / WAVES) + 4 * g4;
    f32x4 kf[2][CQ], ge[KDA ? 2 : 1][CQ];
    float gs[2], dx[2][EG];
    int bs[2], bhi[2];  // the blocks' streams, one past their newest entries
    // lane c16: the c16-th newest entry of a block
    const auto load_keys = [&](int p, int blk) {
        block_at(blk, bs[p], bhi[p]);
        const int e = bhi[p] - 1 - c16;
        const int64_t at = (int64_t)(b0 + bs[p]) * cap + (e > 0 ? e : 0);
        const float *kp = a.tape.k + (at * Hqk + hq) * DK + wc;
#pragma unroll
        for (int i = 0; i < CQ; ++i)
            kf[p][i] = load4(kp + 16 * i);
        if constexpr (KDA) {
            const float *gp = a.tape.g + (at * H + head) * DK + wc;
#pragma unroll
            for (int i = 0; i < CQ; ++i)
                ge[p][i] = load4(gp + 16 * i);
        } else if (wave == 0)
            gs[p] = a.tape.g[at * H + head];
    };
    const auto load_updates = [&](int p) {
        const float *dp = a.tape.d + (((int64_t)(b0 + bs[p]) * cap + bhi[p] - 1) * H + head) * DV + col;
#pragma unroll
        for (int i = 0; i < EG; ++i) {
            const int e = grp * EG + i;  // the block's e-th newest entry
            dx[p][i] = e < bhi[p] ? dp[-(int64_t)e * H * DV] : 0.f;
        }
    };
#pragma unroll
    for (int p = 0; p < 2; ++p) {
        bs[p] = 0, bhi[p] = 1;
        if (p < nblk) {
            load_keys(p, p);
            load_updates(p);
        }
    }

    // ---- front end ---------------------------------------------------------------------------
    if (tid >= THREADS - TOK) {
        const int tok = tid - (THREADS - TOK), s = stream_of(tok);
        bet[tok] = bet_r;
        if constexpr (!KDA) {  // the log-gates through each token, and the tape's
            float sum = 0.f;
#pragma unroll
            for (int j = 0; j < TOK; ++j) {
                const float gj = __builtin_bit_cast(
                    float, __builtin_amdgcn_readlane(__builtin_bit_cast(int, g_r), 64 - TOK + j));
                sum += j >= s * Tn && j <= tok ? gj : 0.f;
            }
            gam[tok] = sum;
            int n = -1;
#pragma unroll
            for (int i = 0; i < NS; ++i) {  // by readlane: the other lanes are not in here
                const int ni = tape_len(i);
                n = s == i ? ni : n;
            }
            if (tok < nt && n >= 0)
                a.tape.g[((int64_t)(b0 + s) * cap + n + tok - s * Tn) * H + head] = g_r;
        }
    }
    if constexpr (KDA) {
#pragma unroll
        for (int p = 0; p < GL; ++p)
            if (tid + p * THREADS < TOK * DK / 4)
                *(f32x4 *)(gk + 4 * (tid + p * THREADS)) = g4r[p];
    }
    for (int i = tid; i < NS * GW; i += THREADS)
        run[i] = 0.f;
    if (tid < CP) {
        float *dst = sec == 2 ? vd + fe : kq + (sec == 0 ? TOK * LDK : 0) + fe;
        const int ldd = sec == 2 ? DV : LDK;
        float2 win[W > 0 ? W : 1];
        T *put = nullptr;
        int s = 0, t = 0;
#pragma unroll
        for (int tok = 0; tok < TOK; ++tok) {
            float x0 = P::lo(raw[tok]), x1 = P::hi(raw[tok]);
            if (K > 0 && tok < nt) {
                if (t == 0) {
                    const int n = tape_len(s);
                    put = n >= 0 && (sec == 2 || own_qk)
                              ? (T *)a.tape.raw + ((int64_t)(b0 + s) * cap + n) * cd + ch
                              : nullptr;
#pragma unroll
                    for (int i = 0; i < W; ++i)
                        win[i] = float2{P::lo(old[tok][i]), P::hi(old[tok][i])};
                }
                float a0 = w[K > 0 ? K - 1 : 0].x * x0, a1 = w[K > 0 ? K - 1 : 0].y * x1;
#pragma unroll
                for (int i = 0; i < W; ++i)
                    a0 += w[i].x * win[i].x, a1 += w[i].y * win[i].y;
#pragma unroll
                for (int i = 0; i + 1 < W; ++i)
                    win[i] = win[i + 1];
                win[W > 0 ? W - 1 : 0] = float2{x0, x1};
                x0 = silu(a0), x1 = silu(a1);
                if (put)
                    *(typename P::raw *)(put + t * cd) = raw[tok];
                if (++t == Tn)
                    t = 0, ++s;
            }
            *(float2 *)(dst + tok * ldd) = float2{x0, x1};
        }
    }
    __syncthreads();

    // ---- L2 and scale: 16 lanes per row; the new entries' keys ------------------------------
#pragma unroll
    for (int m0 = 0; m0 < R; m0 += THREADS / 16) {
        const int m = m0 + (tid >> 4), tok = m % TOK, l = tid & 15;
        float *x = kq + m * LDK + 4 * l;
        f32x4 v[DK / 64];
        float ss = 0.f;
#pragma unroll
        for (int i = 0; i < DK / 64; ++i) {
            v[i] = load4(x + 64 * i);
            ss += v[i].x * v[i].x + v[i].y * v[i].y + v[i].z * v[i].z + v[i].w * v[i].w;
        }
        ss = row_sum(ss);
        float mul = a.do_l2 ? __builtin_amdgcn_rsqf(ss + a.eps) : 1.f;
        if (m >= TOK)
            mul *= a.scale;
        const int s = stream_of(tok), n = tok < nt ? slen[s] : -1;
#pragma unroll
        for (int i = 0; i < DK / 64; ++i) {
            v[i] = tok < nt ? v[i] * mul : zero4();
            *(f32x4 *)(x + 64 * i) = v[i];
            if (m < TOK && own_qk && n >= 0)
                *(f32x4 *)(a.tape.k + (((int64_t)(b0 + s) * cap + n + tok - s * Tn) * Hqk + hq) * DK +
                           4 * l + 64 * i) = v[i];
        }
    }
    // KDA: running sums of the log-gates within each stream's new tokens; their tape entries
    if constexpr (KDA) {
        if (tid < DK) {
            float gv[TOK];
#pragma unroll
            for (int tok = 0; tok < TOK; ++tok)
                gv[tok] = gk[tok * DK + tid];
            int s = 0, t = 0, n = 0;
            float sum = 0.f;
#pragma unroll
            for (int tok = 0; tok < TOK; ++tok) {
                if (tok < nt) {
                    if (t == 0)
                        n = tape_len(s), sum = 0.f;
                    if (n >= 0)
                        a.tape.g[(((int64_t)(b0 + s) * cap + n + t) * H + head) * DK + tid] = gv[tok];
                    sum += gv[tok];
                    gk[tok * DK + tid] = sum;
                    if (++t == Tn)
                        t = 0, ++s;
                }
            }
        }
    }
    __syncthreads();

    // ---- coefficients among the new tokens: 16 lanes per pair (x, y) of a stream's tokens:
    // y < x: key y in d_x; y >= x: key x in o_y --------------------------------------------
    {
        const int per = Tn * Tn, inv_p = (65536 + per - 1) / per, inv_x = (65536 + Tn - 1) / Tn, l = tid & 15;
        for (int idx = tid >> 4; idx < ns * per; idx += THREADS / 16) {
            const int s = idx * inv_p >> 16, r = idx - s * per, xx = r * inv_x >> 16, yy = r - xx * Tn;
            const int tok = s * Tn + (yy < xx ? xx : yy), j = s * Tn + (yy < xx ? yy : xx);
            const int u = yy < xx ? xx : yy, m = (yy < xx ? 0 : TOK) + tok;
            float sum = 0.f;
#pragma unroll
            for (int i = 0; i < DK / 64; ++i) {
                const f32x4 x = load4(kq + m * LDK + 4 * l + 64 * i);
                f32x4 kj = load4(kq + j * LDK + 4 * l + 64 * i);
                if constexpr (KDA) {
                    const f32x4 e = load4(gk + tok * DK + 4 * l + 64 * i) - load4(gk + j * DK + 4 * l + 64 * i);
                    kj *= f32x4{__expf(e.x), __expf(e.y), __expf(e.z), __expf(e.w)};
                }
                sum += x.x * kj.x + x.y * kj.y + x.z * kj.z + x.w * kj.w;
            }
            sum = row_sum(sum);
            if constexpr (!KDA)
                sum *= __expf(gam[tok] - gam[j]);
            if (l == 0)
                co[((yy < xx ? 0 : TOK) + j) * TOK + u] = sum;  // by entry j, then token u
        }
    }
    if constexpr (KDA) {  // keys and queries take the decay through their token
        __syncthreads();
        for (int i = tid; i < R * (DK / 4); i += THREADS) {
            const int m = i / (DK / 4), c = 4 * (i % (DK / 4)), tok = m % TOK;
            if (tok < nt) {
                const f32x4 e = load4(gk + tok * DK + c);
                float *x = kq + m * LDK + c;
                *(f32x4 *)x = load4(x) * f32x4{__expf(e.x), __expf(e.y), __expf(e.z), __expf(e.w)};
            }
        }
    }

    // ---- the tapes, two blocks a round: each wave's channels of their scores against all
    // rows, summed over the waves; then a thread per column adds the blocks' updates to the
    // rows of their own streams (so what a tape holds reaches no other stream, be it NaN) ------
    float hist[R];
#pragma unroll
    for (int m = 0; m < R; ++m)
        hist[m] = 0.f;
    if (KDA && nblk > 0)
        __syncthreads();  // the decayed keys and queries
    for (int blk0 = 0; blk0 < nblk; blk0 += 2) {
#pragma unroll
        for (int p = 0; p < 2; ++p) {
            if (blk0 + p >= nblk)
                continue;
            // the decay after each entry: over the block's newer entries (a scan over the
            // lanes) and over the tape's newer blocks
            const bool in = bhi[p] - 1 - c16 >= 0;
            if constexpr (KDA) {
                float *const rp = run + bs[p] * DK + wc;
#pragma unroll
                for (int i = 0; i < CQ; ++i) {
                    const f32x4 newer = load4(rp + 16 * i);
                    f32x4 sum;
#pragma unroll
                    for (int j = 0; j < 4; ++j) {
                        sum[j] = row_scan(in ? ge[p][i][j] : 0.f);
                        kf[p][i][j] *= __expf(dpp<DPP_SHR + 1>(sum[j]) + newer[j]);
                    }
                    if (c16 == 15)  // this wave alone reads and writes these channels
                        *(f32x4 *)(rp + 16 * i) = newer + sum;
                }
            } else if (wave == 0) {
                const float sum = row_scan(in ? gs[p] : 0.f), newer = run[bs[p]];
                if (g4 == 0)
                    suf[16 * p + c16] = dpp<DPP_SHR + 1>(sum) + newer;
                if (lane == 15)  // this wave alone writes the sums, and reads them until the state
                    run[bs[p]] = newer + sum;
            }
            f32x4 sc[MT];
#pragma unroll
            for (int mt = 0; mt < MT; ++mt)
                sc[mt] = zero4();
#pragma unroll
            for (int i = 0; i < CQ; ++i)
#pragma unroll
                for (int mt = 0; mt < MT; ++mt) {
                    const f32x4 av = load4(kq + (16 * mt + c16) * LDK + wc + 16 * i);
#pragma unroll
                    for (int j = 0; j < 4; ++j)
                        sc[mt] = mfma4(av[j], kf[p][i][j], sc[mt]);
                }
#pragma unroll
            for (int mt = 0; mt < MT; ++mt)
#pragma unroll
                for (int r = 0; r < 4; ++r)
                    sp[((p * WAVES + wave) * R + 16 * mt + 4 * g4 + r) * S::LDS_ + c16] = sc[mt][r];
        }
        const int s2[2] = {bs[0], bs[1]}, hi2[2] = {bhi[0], bhi[1]};
#pragma unroll
        for (int p = 0; p < 2; ++p)
            if (blk0 + 2 + p < nblk)
                load_keys(p, blk0 + 2 + p);
        __syncthreads();
#pragma unroll
        for (int i = 0; i < 2 * R * 16 / THREADS; ++i) {
            const int idx = tid + i * THREADS, e = idx & 15, m = idx / 16 % R, p = idx / (16 * R), tok = m % TOK;
            float v = 0.f;
#pragma unroll
            for (int q = 0; q < WAVES; ++q)
                v += sp[((p * WAVES + q) * R + m) * S::LDS_ + e];
            if constexpr (!KDA)
                v *= __expf(gam[tok] + suf[16 * p + e]);
            fs[(p * R + m) * S::LDS_ + e] = e < (p ? hi2[1] : hi2[0]) ? v : 0.f;
        }
        __syncthreads();
#pragma unroll
        for (int p = 0; p < 2; ++p) {
            if (blk0 + p >= nblk)
                continue;
            const int lo = s2[p] * Tn, up = lo + Tn;
            const float *xp = fs + p * R * S::LDS_ + grp * EG;
#pragma unroll
            for (int m = 0; m < TOK; ++m) {
                if (m < lo || m >= up)
                    continue;
#pragma unroll
                for (int i = 0; i < EG; i += 4) {
                    const f32x4 xk = load4(xp + m * S::LDS_ + i), xq = load4(xp + (TOK + m) * S::LDS_ + i);
#pragma unroll
                    for (int j = 0; j < 4; ++j) {
                        hist[m] += xk[j] * dx[p][i + j];
                        hist[TOK + m] += xq[j] * dx[p][i + j];
                    }
                }
            }
        }
#pragma unroll
        for (int p = 0; p < 2; ++p)
            if (blk0 + 2 + p < nblk)
                load_updates(p);
    }
    if (nblk > 0)
        __syncthreads();

    // ---- the state, 64 columns and RW rows per wave: lane (g4, c16) loads 4 adjacent columns
    // of the rows 4 g4 + i, which serve 4 products of 16 columns each ------------------------
    {
        f32x4 hr[S::RW / 4], acc[MT][4];
        const float *hp = a.h_ptrs[pfx] + (int64_t)head * DK * DV +
                          (int64_t)(rs * S::RW + 4 * g4) * DV + 64 * cg + 4 * c16;
#pragma unroll
        for (int i = 0; i < S::RW / 4; ++i)
            hr[i] = load_nt4(hp + (int64_t)(16 * (i / 4) + i % 4) * DV);
        // the products start from what the tapes gave: part grp of a column's threads
        float *const yp = y + (rs * R + 4 * g4) * DV + 64 * cg + 4 * c16;
        if (nblk > 0) {
#pragma unroll
            for (int m = 0; m < R; ++m)
                y[(grp * R + m) * DV + col] = hist[m];
        }
        __syncthreads();
        float f[MT];
#pragma unroll
        for (int mt = 0; mt < MT; ++mt) {
            const int tok = (16 * mt + c16) % TOK;
            f[mt] = 1.f;
            if constexpr (!KDA)
                f[mt] = tok < nt ? __expf(gam[tok] + run[stream_of(tok)]) : 0.f;
            f32x4 v[4];
#pragma unroll
            for (int r = 0; r < 4; ++r)
                v[r] = nblk > 0 ? load4(yp + (16 * mt + r) * DV) : zero4();
#pragma unroll
            for (int j = 0; j < 4; ++j)
                acc[mt][j] = f32x4{v[0][j], v[1][j], v[2][j], v[3][j]};
        }
#pragma unroll
        for (int ss = 0; ss < S::RW / 16; ++ss) {
            const int c = rs * S::RW + 16 * ss + 4 * g4;
            f32x4 av[MT];
#pragma unroll
            for (int mt = 0; mt < MT; ++mt) {
                const int tok = (16 * mt + c16) % TOK;
                av[mt] = load4(kq + (16 * mt + c16) * LDK + c);
                if constexpr (KDA) {
                    const f32x4 x = load4(run + (tok < nt ? stream_of(tok) : 0) * DK + c);
                    av[mt] *= f32x4{__expf(x.x), __expf(x.y), __expf(x.z), __expf(x.w)};
                } else
                    av[mt] *= f[mt];
            }
#pragma unroll
            for (int i = 0; i < 4; ++i)
#pragma unroll
                for (int mt = 0; mt < MT; ++mt)
#pragma unroll
                    for (int j = 0; j < 4; ++j)
                        acc[mt][j] = mfma4(av[mt][i], hr[4 * ss + i][j], acc[mt][j]);
        }
#pragma unroll
        for (int mt = 0; mt < MT; ++mt)
#pragma unroll
            for (int r = 0; r < 4; ++r)
                *(f32x4 *)(yp + (16 * mt + r) * DV) =
                    f32x4{acc[mt][0][r], acc[mt][1][r], acc[mt][2][r], acc[mt][3][r]};
    }
    __syncthreads();

    // ---- the new tokens in order, a thread per column ------------------------------------
    for (int s = grp; s < ns; s += S::G) {
        const int n = tape_len(s);
        if (n < 0)
            continue;
        const int lo = s * Tn;
        float yk[TOK], yq[TOK], v[TOK], bb[TOK];
#pragma unroll
        for (int t = 0; t < TOK; ++t) {
            const int tok = lo + (t < Tn ? t : 0);  // rows past the stream's: of no use
            yk[t] = y[tok * DV + col], yq[t] = y[(TOK + tok) * DV + col];
#pragma unroll
            for (int p = 1; p < S::RS; ++p) {
                yk[t] += y[(p * R + tok) * DV + col];
                yq[t] += y[(p * R + TOK + tok) * DV + col];
            }
            v[t] = vd[tok * DV + col];
            bb[t] = bet[tok];
        }
        float *dp = a.tape.d + (((int64_t)(b0 + s) * cap + n) * H + head) * DV + col;
        float *op = a.o + ((row0 + lo) * H + head) * DV + col;
#pragma unroll
        for (int t = 0; t < TOK; ++t) {
            if (t >= Tn)
                continue;
            f32x4 ck[TOK / 4], cq[TOK / 4];
#pragma unroll
            for (int u = 0; u < TOK / 4; ++u) {
                ck[u] = load4(co + (lo + t) * TOK + 4 * u);
                cq[u] = load4(co + (TOK + lo + t) * TOK + 4 * u);
            }
            const float d = bb[t] * (v[t] - yk[t]);
            dp[(int64_t)t * H * DV] = d;
#pragma unroll
            for (int u = t; u < TOK; ++u) {  // coefficients of tokens past T: of no use
                if (u > t)
                    yk[u] += ck[u / 4][u % 4] * d;
                yq[u] += cq[u / 4][u % 4] * d;
            }
            if (a.z)
                y[(TOK + lo + t) * DV + col] = yq[t];
            else
                op[(int64_t)t * H * DV] = yq[t];
        }
    }
    if (!a.z)
        return;
    __syncthreads();

    // ---- o through the output gate -------------------------------------------------------
    constexpr int L = DV / 4;
    for (int tok = tid / L; tok < nt; tok += THREADS / L) {
        const int l = tid % L;
        if (slen[stream_of(tok)] < 0)
            continue;
        f32x4 o = load4(y + (TOK + tok) * DV + 4 * l);
        const f32x4 z = load4((const T *)a.z + (row0 + tok) * a.ld_z + (int64_t)head * DV + 4 * l);
        const f32x4 w = load4(a.norm_w + 4 * l);
        const float ss = group_sum<L>(o.x * o.x + o.y * o.y + o.z * o.z + o.w * o.w);
        const float inv = __builtin_amdgcn_rsqf(ss * (1.f / DV) + a.norm_eps);
#pragma unroll
        for (int i = 0; i < 4; ++i)
            o[i] *= inv * w[i] * silu(z[i]);
        *(f32x4 *)(a.o + ((row0 + tok) * H + head) * DV + 4 * l) = o;
    }
}

// One workgroup: SL columns of one stream and head's state, held in MFMA accumulator layout:
// lane (g4, c16) has rows 16*rt + 4*g4 + r and 4 adjacent columns of the wave's 64. The tape
// is taken in blocks of 16 entries, oldest first: the state times the block's decay, plus the
// block's entries with the decay after each (summed from the newest back: no differences of
// long sums). A block's loads go out while the one before is worked in.
//
// The accumulators cross the loop's edges; the wait states that an MFMA result needs before
// another instruction reads it are kept there by hand (settle), since along a branch the
// compiler has placed too few of them before.
__device__ __forceinline__ void settle()
{
    __builtin_amdgcn_sched_barrier(0);
    asm volatile("s_nop 7\n\ts_nop 7");
    __builtin_amdgcn_sched_barrier(0);
}

template <typename T, int DK, int DV, bool KDA, int SL>
__global__ void __launch_bounds__(THREADS, SL == 64 ? 4 : 3) fold_kernel(const FoldArgs a)
{
    constexpr int CG = SL / 64, RS = WAVES / CG, RW = DK / RS, RT = RW / 16;
    constexpr int EB = 16;                              // tape entries per block
    constexpr int GW = KDA ? DK : 1;                    // log-gates per entry
    constexpr int GP = KDA ? THREADS / DK : 1;          // threads per log-gate column
    static_assert(RT >= 1 && EB % GP == 0, "tile map");
    __shared__ __align__(16) float sf[2][EB * GW];      // decay after each entry
    __shared__ __align__(16) float through[2][GW];      // decay of the block

    const int H = a.H, Hqk = a.Hqk, cap = a.tape.cap;
    const int bh = blockIdx.x / (DV / SL), slice = blockIdx.x % (DV / SL);
    const int b = bh / H, head = bh % H, pfx = b / a.share;
    const int rep = H / Hqk, hq = head / rep;
    const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
    const int c16 = lane & 15, g4 = lane >> 4;
    const int cg = wave % CG, rs = wave / CG;
    const int n = a.tape.len[b];
    const bool bad = n < 0 || n > cap;
    const bool on = !bad && n >= a.min_len;
    if (head == 0 && slice == 0 && tid == 0) {
        if (bad && a.tape.status)
            atomicOr(a.tape.status, GDN_BAD_TAPE);
        if (a.len_out && a.len_out != a.tape.len)
            a.len_out[b] = on ? 0 : n;
    }
    if (!on)
        return;

    const int64_t e0 = (int64_t)b * cap;
    // a block's log-gates: all threads of a column have all 16
    const int gc = tid % GW, gp = tid / GW;
    const float *gp0 = a.tape.g + (e0 * H + head) * GW + gc;
    const int64_t ge = (int64_t)H * GW;
    float gv[EB];
    const auto load_gates = [&](int eb) {
#pragma unroll
        for (int e = 0; e < EB; ++e)
            gv[e] = eb + e < n ? gp0[(eb + e) * ge] : 0.f;
    };
    // its updates and keys: lane g4 takes entries g4, 4 + g4, ...
    f32x4 dv[EB / 4];
    float kv[EB / 4][RT];
    const auto load_entries = [&](int eb) {
#pragma unroll
        for (int q = 0; q < EB / 4; ++q) {
            const int e = eb + 4 * q + g4;
            const bool in = e < n;
            const int64_t at = e0 + (in ? e : 0);
            const f32x4 d = load4(a.tape.d + (at * H + head) * DV + SL * slice + 64 * cg + 4 * c16);
            dv[q] = in ? d : zero4();
#pragma unroll
            for (int rt = 0; rt < RT; ++rt) {
                const float k = a.tape.k[(at * Hqk + hq) * DK + rs * RW + 16 * rt + c16];
                kv[q][rt] = in ? k : 0.f;
            }
        }
    };
    if (gp < GP)
        load_gates(0);
    load_entries(0);
    const int64_t hoff = (int64_t)head * DK * DV + (int64_t)(rs * RW + 4 * g4) * DV + SL * slice +
                         64 * cg + 4 * c16;
    const float *hp = a.h_ptrs[pfx] + hoff;
    f32x4 acc[RT][4];  // [row tile][column of 4]: rows r
#pragma unroll
    for (int rt = 0; rt < RT; ++rt) {
        f32x4 hr[4];
#pragma unroll
        for (int r = 0; r < 4; ++r)
            hr[r] = load_nt4(hp + (int64_t)(16 * rt + r) * DV);
#pragma unroll
        for (int j = 0; j < 4; ++j)
            acc[rt][j] = f32x4{hr[0][j], hr[1][j], hr[2][j], hr[3][j]};
    }

    // the windows after the tape: the last K-1 raw inputs of the channels of this head (those
    // of a q/k head by its first value head)
    if (a.K > 0 && slice == 0) {
        const int W = a.K - 1;
        const int64_t cd = 2 * (int64_t)Hqk * DK + (int64_t)H * DV;
        const T *in = (const T *)a.conv_state_ptrs[pfx];
        T *out = (T *)a.conv_out_ptrs[b];
        for (int c = tid; c < 2 * DK + DV; c += THREADS) {
            if (c < 2 * DK && head % rep)
                continue;
            const int64_t ch = c < DK       ? (int64_t)hq * DK + c
                               : c < 2 * DK ? (int64_t)(Hqk + hq) * DK + c - DK
                                            : 2 * (int64_t)Hqk * DK + (int64_t)head * DV + c - 2 * DK;
            T w[3];
#pragma unroll
            for (int i = 0; i < 3; ++i) {
                const int m = n - W + i;
                if (i < W)
                    w[i] = m >= 0 ? ((const T *)a.tape.raw)[(e0 + m) * cd + ch] : in[ch * W + W + m];
            }
#pragma unroll
            for (int i = 0; i < 3; ++i)
                if (i < W)
                    out[ch * W + i] = w[i];
        }
    }

    for (int eb = 0, buf = 0; eb < n; eb += EB, buf ^= 1) {
        if (gp < GP) {
            float run = 0.f;
#pragma unroll
            for (int e = EB - 1; e >= 0; --e) {
                if (e % GP == gp)
                    sf[buf][e * GW + gc] = __expf(run);
                run += gv[e];
            }
            if (gp == 0)
                through[buf][gc] = __expf(run);
            if (eb + EB < n)
                load_gates(eb + EB);
        }
        __syncthreads();  // one per block: its factors lie in the buffer of the one before last
#pragma unroll
        for (int rt = 0; rt < RT; ++rt)
#pragma unroll
            for (int r = 0; r < 4; ++r) {
                const float f = through[buf][KDA ? rs * RW + 16 * rt + 4 * g4 + r : 0];
#pragma unroll
                for (int j = 0; j < 4; ++j)
                    acc[rt][j][r] *= f;
            }
#pragma unroll
        for (int q = 0; q < EB / 4; ++q)
#pragma unroll
            for (int rt = 0; rt < RT; ++rt) {
                const float k = kv[q][rt] * sf[buf][(4 * q + g4) * GW + (KDA ? rs * RW + 16 * rt + c16 : 0)];
#pragma unroll
                for (int j = 0; j < 4; ++j)
                    acc[rt][j] = mfma4(k, dv[q][j], acc[rt][j]);
            }
        settle();
        if (eb + EB < n)
            load_entries(eb + EB);
    }
    float *op = a.h_out_ptrs[b] + hoff;
#pragma unroll
    for (int rt = 0; rt < RT; ++rt)
#pragma unroll
        for (int r = 0; r < 4; ++r)
            __builtin_nontemporal_store(f32x4{acc[rt][0][r], acc[rt][1][r], acc[rt][2][r], acc[rt][3][r]},
                                        (f32x4 *)(op + (int64_t)(16 * rt + r) * DV));
}

// tape lengths after a fold that was asked to clear them in place
__global__ void __launch_bounds__(THREADS) fold_len_kernel(int32_t *len, int32_t B, int32_t cap, int32_t min_len)
{
    const int b = blockIdx.x * THREADS + threadIdx.x;
    if (b < B && len[b] <= cap && len[b] >= min_len)
        len[b] = 0;
}

template <typename T, int DK, int DV, bool KDA, int TOK>
hipError_t draft_k(const DraftArgs &a, hipStream_t s)
{
    using S = DraftShape<DK, DV, KDA, TOK>;
    const int ns = TOK / a.T < S::NS ? TOK / a.T : S::NS;
    const int ntile = (a.share + ns - 1) / ns;
    const int64_t grid = ((int64_t)(a.B / a.share) * a.H + 7) / 8 * 8 * ntile;
    if (grid > (int64_t)INT32_MAX)
        return hipErrorInvalidValue;
    const dim3 g((unsigned)grid), t(THREADS);
    switch (a.K) {
    case 0: hipLaunchKernelGGL((draft_kernel<T, DK, DV, KDA, 0, TOK>), g, t, 0, s, a, ntile); break;
    case 2: hipLaunchKernelGGL((draft_kernel<T, DK, DV, KDA, 2, TOK>), g, t, 0, s, a, ntile); break;
    case 3: hipLaunchKernelGGL((draft_kernel<T, DK, DV, KDA, 3, TOK>), g, t, 0, s, a, ntile); break;
    case 4: hipLaunchKernelGGL((draft_kernel<T, DK, DV, KDA, 4, TOK>), g, t, 0, s, a, ntile); break;
    default: return hipErrorInvalidValue;
    }
    return hipGetLastError();
}

template <typename T, int DK, int DV, bool KDA> hipError_t draft_t(const DraftArgs &a, hipStream_t s)
{
    return a.T <= 8 ? draft_k<T, DK, DV, KDA, 8>(a, s) : draft_k<T, DK, DV, KDA, 16>(a, s);
}

template <typename T, int DK, int DV, bool KDA, int SL> hipError_t fold_s(const FoldArgs &a, hipStream_t s)
{
    const int64_t grid = (int64_t)a.B * a.H * (DV / SL);
    if (grid > (int64_t)INT32_MAX)
        return hipErrorInvalidValue;
    hipLaunchKernelGGL((fold_kernel<T, DK, DV, KDA, SL>), dim3((unsigned)grid), dim3(THREADS), 0, s, a);
    if (hipError_t e = hipGetLastError(); e != hipSuccess)
        return e;
    if (a.len_out == a.tape.len)
        hipLaunchKernelGGL(fold_len_kernel, dim3((unsigned)((a.B + THREADS - 1) / THREADS)), dim3(THREADS), 0, s,
                           a.tape.len, a.B, a.tape.cap, a.min_len);
    return hipGetLastError();
}

template <typename T, int DK, int DV, bool KDA> hipError_t fold_t(const FoldArgs &a, hipStream_t s)
{
    // Slices of 64 columns at 4 waves per SIMD (64 x 32 heads: 57.5 us, whole rows of 128 columns
    // 61.8 us; 1 x 32 heads: 6.4 us and 8.8 us), but for many channel-gated heads, whose factors
    // each slice forms again (48 x 32 heads: slices 48 us, whole rows 44 us).
    if (KDA && DV > 64 && (int64_t)a.B * a.H >= 1024)
        return fold_s<T, DK, DV, KDA, DV < 128 ? DV : 128>(a, s);
    return fold_s<T, DK, DV, KDA, 64>(a, s);
}

// f<T, DK, DV, KDA>(a, s) for the compiled configurations: bf16 (64, 64), (128, 128) and
// (128, 256), float32 (64, 64) and (64, 128)
#define GDN_DISPATCH(F, a, s)                                                                   \
    if (dtype) {                                                                                \
        if ((a).dk == 128 && (a).dv == 128)                                                     \
            return kda ? F<bf16, 128, 128, true>(a, s) : F<bf16, 128, 128, false>(a, s);        \
        if ((a).dk == 128 && (a).dv == 256)                                                     \
            return kda ? F<bf16, 128, 256, true>(a, s) : F<bf16, 128, 256, false>(a, s);        \
        if ((a).dk == 64 && (a).dv == 64)                                                       \
            return kda ? F<bf16, 64, 64, true>(a, s) : F<bf16, 64, 64, false>(a, s);            \
    } else {                                                                                    \
        if ((a).dk == 64 && (a).dv == 64)                                                       \
            return kda ? F<float, 64, 64, true>(a, s) : F<float, 64, 64, false>(a, s);          \
        if ((a).dk == 64 && (a).dv == 128)                                                      \
            return kda ? F<float, 64, 128, true>(a, s) : F<float, 64, 128, false>(a, s);        \
    }                                                                                           \
    return hipErrorInvalidValue

}  // namespace

hipError_t launch_draft(int dtype, int kda, const DraftArgs &a, hipStream_t s)
{
    GDN_DISPATCH(draft_t, a, s);
}

hipError_t launch_fold(int dtype, int kda, const FoldArgs &a, hipStream_t s)
{
    GDN_DISPATCH(fold_t, a, s);
}

}  // namespace gdn
