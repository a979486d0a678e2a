// Sequence-wise balance loss (a training-side quantity beside the routing).
//
// "DeepSeek-V3 Technical Report" notes, bias paragraph: besides the bias, a
// very small sequence-wise loss guards against extreme imbalance inside one
// sequence.  The pages give no formula; this library's reading is the usual
// frequency-times-probability balance term, per sequence of L tokens:
//     f_i  = E / (K L) * #{tokens of the sequence that chose expert i}
//     P_i  = (1/L) * sum_t s[t,i] / sum_j s[t,j]      (raw sigmoid scores)
//     loss = alpha * sum_i f_i P_i
// Uniform use gives alpha; every token on the same K experts with all of its
// score on them gives alpha * E / K.  A token whose scores sum to 0 adds
// nothing to P.
//
// Two passes, both in a fixed order (deterministic).  Pass 1: one block of 4
// waves per chunk of 64 tokens of a sequence; wave w takes tokens w, w+4, ...
// of the chunk, four rows at a time so that four row loads are in flight;
// lane l holds experts l, l+64, l+128, l+192; per token the wave sums the row
// (each lane over its experts in order, then a butterfly), divides and
// accumulates.  Expert counts go to LDS with integer atomics (exact in any
// order).  The chunk's partial P and counts go to the workspace.  Pass 2: one
// block per sequence adds the chunks in order and reduces the E terms by a
// fixed tree.
#include <limits.h>

#include "kernels.h"
#include "lanes.h"
#include "streaming.h"

namespace moe {
namespace {

constexpr int BAL_CHUNK = 64;       // tokens per pass-1 block
constexpr int BAL_WAVES = 4;
constexpr int BAL_UNROLL = 4;       // rows in flight per wave

struct BalancePart {
    float p[256];
    int32_t cnt[256];
};

__global__ __launch_bounds__(64 * BAL_WAVES) void seq_balance_partial_kernel(
    const float* __restrict__ s, const int32_t* __restrict__ idx, int E, int K, int L, int nchunk,
    BalancePart* __restrict__ part) {
    __shared__ int cnt[256];
    __shared__ float wpart[BAL_WAVES][256];
    const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
    cnt[tid] = 0;                                   // 256 threads
    __syncthreads();
    const int q = blockIdx.x / nchunk, c = blockIdx.x % nchunk;
    const int tb = c * BAL_CHUNK, te = min(L, tb + BAL_CHUNK);
    const int64_t base = (int64_t)q * L;
    float acc[4] = {0.f, 0.f, 0.f, 0.f};
    for (int t = tb + wave; t < te; t += BAL_WAVES * BAL_UNROLL) {
        float v[BAL_UNROLL][4];
#pragma unroll
        for (int r = 0; r < BAL_UNROLL; ++r) {
            const int tt = t + r * BAL_WAVES;
            const float* row = s + (base + tt) * E;
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const int e = lane + 64 * j;
                v[r][j] = (tt < te && e < E) ? row[e] : 0.f;
            }
        }
#pragma unroll
        for (int r = 0; r < BAL_UNROLL; ++r) {
            float rs = 0.f;
#pragma unroll
            for (int j = 0; j < 4; ++j) rs = rs + v[r][j];
#pragma unroll
            for (int off = 1; off < 64; off <<= 1) rs = rs + __shfl_xor(rs, off, 64);
            if (rs != 0.f) {
#pragma unroll
                for (int j = 0; j < 4; ++j) acc[j] = acc[j] + v[r][j] / rs;
            }
            const int tt = t + r * BAL_WAVES;
            if (tt < te && lane < K) {
                const int e = idx[(base + tt) * K + lane];
                if ((unsigned)e < (unsigned)E) atomicAdd(&cnt[e], 1);     // other values are ignored
            }
        }
    }
#pragma unroll
    for (int j = 0; j < 4; ++j) wpart[wave][lane + 64 * j] = acc[j];
    __syncthreads();
    float p = 0.f;
#pragma unroll
    for (int w = 0; w < BAL_WAVES; ++w) p = p + wpart[w][tid];
    part[blockIdx.x].p[tid] = p;
    part[blockIdx.x].cnt[tid] = cnt[tid];
}

__global__ __launch_bounds__(256) void seq_balance_final_kernel(const BalancePart* __restrict__ part,
                                                                int E, int K, int L, int nchunk,
                                                                float alpha, float* __restrict__ loss) {
    __shared__ float term[256];
    const int tid = threadIdx.x, q = blockIdx.x;
    float p = 0.f;
    int n = 0;
    for (int c = 0; c < nchunk; ++c) {
        p = p + part[(int64_t)q * nchunk + c].p[tid];
        n += part[(int64_t)q * nchunk + c].cnt[tid];
    }
    const float f = (float)E * (float)n / ((float)K * (float)L);
    term[tid] = tid < E ? f * (p / (float)L) : 0.f;
    __syncthreads();
    for (int h = 128; h >= 1; h >>= 1) {
        if (tid < h) term[tid] = term[tid] + term[tid + h];
        __syncthreads();
    }
    if (tid == 0) loss[q] = alpha * term[0];
}

// ---------------------------------------------------------------------------
// The same loss over sequences of any lengths, with the counts that the gradient
// and the bias update take, and its gradient with respect to the router's logits.
// Sequence q holds the tokens [start[q], start[q+1]); with p = s / sum_j s_j,
//     f_i = E n_i / (K L),  P_i = (1/L) sum_t p_ti,  loss_q = alpha sum_i f_i P_i,
//     dlogit_ti = dloss_q alpha / L * p_ti (1 - s_ti) (f_i - sum_j f_j p_tj)
// (the counts n are held fixed; s' = s (1 - s)).
//
// Forward.  Block c takes the tokens [c chunk, (c+1) chunk), one run of them for
// each sequence that the chunk meets, and leaves the run's partial sums of p and
// its counts as record c + q: along the chunks and sequences that meet, c + q grows
// at every step, so no two runs share a record.  The chunk's counts over its runs
// are kept too.  A second launch adds up each sequence's records, and the chunks'
// counts.  Small calls take one launch, a block to a sequence.  Every order is fixed by the sizes and the starts.

constexpr int RUN_WAVES = 16;
constexpr int RUN_CHUNKS = 256;     // at most: one block per CU
constexpr int RUN_LEAST = 64;       // tokens of a chunk at least

// start[i], held inside [0, T]; without an array one sequence of all T tokens
__device__ __forceinline__ int seq_start_at(const int32_t* __restrict__ start, int i, int n_seq, int T) {
    if (!start) return i < n_seq ? 0 : T;
    return min(max(start[i], 0), T);
}

// The first sequence that ends behind token t (n_seq if none does): LPT lanes, who all
// want the same, look at LPT ends at a time.
template <int LPT>
__device__ __forceinline__ int seq_of(const int32_t* __restrict__ start, int n_seq, int T, int t) {
    const int l = threadIdx.x % LPT, shift = (threadIdx.x & 63) / LPT * LPT;
    int lo = 0, hi = n_seq;
    while (lo < hi) {
        const int step = (hi - lo + LPT - 1) / LPT, at = lo + (l + 1) * step - 1;
        const uint64_t ends = __ballot(at >= hi || seq_start_at(start, at + 1, n_seq, T) > t) >> shift;
        const uint64_t mine = LPT == 64 ? ends : ends & 0xFFFFull;
        if (!mine) return hi;
        const int first = __builtin_ctzll(mine);
        hi = min(hi, lo + (first + 1) * step - 1);    // the answer at most, as that one ends behind t
        lo = lo + first * step;
        if (step == 1) return lo;
    }
    return lo;
}

struct BalanceRun {                 // record of a run; [256] each, but a call's own E are in use
    float p[256];
    int32_t n[256];
};

// LPT lanes hold a token, 4 of its experts each: 4 l to 4 l + 3 (VEC: E % 4 == 0), or
// l + LPT j.
template <int LPT, bool VEC>
__device__ __forceinline__ int expert_of(int l, int j) { return VEC ? 4 * l + j : l + LPT * j; }

template <int LPT, bool VEC>
__device__ __forceinline__ void load_experts(const float* row, int l, int E, bool in, float (&v)[4]) {
    if constexpr (VEC) {
        const float4 x = in && 4 * l < E ? *reinterpret_cast<const float4*>(row + 4 * l) : make_float4(0.f, 0.f, 0.f, 0.f);
        v[0] = x.x; v[1] = x.y; v[2] = x.z; v[3] = x.w;
    } else {
#pragma unroll
        for (int j = 0; j < 4; ++j) v[j] = in && l + LPT * j < E ? row[l + LPT * j] : 0.0f;
    }
}

template <int LPT>
__device__ __forceinline__ float token_sum(float s) {
    return LPT == 16 ? sum16(s) : wave_sum(s);
}

// A token's shares p = v / sum v (0 where the sum is), rounded as a division rounds them:
// by the sum's reciprocal, which a step of Newton's makes good to half an ulp, and once
// more by what that leaves of v, which an FMA has exactly.  (Of 10^9 quotients one came out
// another; the product with a rounded reciprocal is off in three of ten.  The same time
// as that one's, whose division took more; with that division and this, 65536 tokens in 2000
// sequences 56 us for 53.)  Sums under 2^-64 are scaled up first, so that the reciprocal
// stays finite.
template <int LPT>
__device__ __forceinline__ void shares(const float (&v)[4], float (&p)[4]) {
    float sum = token_sum<LPT>((v[0] + v[1]) + (v[2] + v[3]));
    const float up = __builtin_fabsf(sum) < 0x1p-64f ? 0x1p64f : 1.0f;
    sum *= up;
    const float near = __builtin_amdgcn_rcpf(sum);
    const float inv = sum == 0.0f ? 0.0f : __builtin_fmaf(__builtin_fmaf(-near, sum, 1.0f), near, near);
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        const float x = v[j] * up, q = x * inv;
        p[j] = __builtin_fmaf(__builtin_fmaf(-q, sum, x), inv, q);
    }
}

constexpr int AT_ONCE = 4;          // tokens whose loads go out together

// Bound by the latency of HBM reads: 131072 x 256 with 8 experts a token in 96 sequences
// 30 us (4.6 TB/s), 16384 x 256 in 4 7.  The next four tokens' loads ahead of the sums,
// four indexes at a time, and 16 lanes a token with 16 values each (half the
// instructions) all leave it at that.

template <int LPT> struct RunLds {
    static constexpr int GROUPS = 64 * RUN_WAVES / LPT, WIDE = 4 * LPT;
    int cnt[256];
    float psum[GROUPS][WIDE];
};

// The sums of the shares p of the tokens [rb, re) of one sequence and their counts, by a
// block of RUN_WAVES waves: thread = expert e < E has them afterwards.
template <int LPT, bool VEC>
__device__ __forceinline__ void run_sums(const float* __restrict__ s, const int32_t* __restrict__ idx, int rb, int re,
                                         int E, int K, RunLds<LPT>& lds, float& sum, int& count) {
    constexpr int GROUPS = RunLds<LPT>::GROUPS;
    const int tid = threadIdx.x, l = tid % LPT, grp = tid / LPT;
    if (tid < 256) lds.cnt[tid] = 0;
    __syncthreads();
    for (int64_t i = (int64_t)rb * K + tid; i < (int64_t)re * K; i += 64 * RUN_WAVES) {
        const int e = idx[i];
        if ((unsigned)e < (unsigned)E) atomicAdd(&lds.cnt[e], 1);          // integers: exact in any order
    }
    float acc[4] = {0.f, 0.f, 0.f, 0.f};
    for (int t = rb + grp; t < re; t += AT_ONCE * GROUPS) {
        float v[AT_ONCE][4];
#pragma unroll
        for (int k = 0; k < AT_ONCE; ++k)
            load_experts<LPT, VEC>(s + (int64_t)(t + k * GROUPS) * E, l, E, t + k * GROUPS < re, v[k]);
#pragma unroll
        for (int k = 0; k < AT_ONCE; ++k) {
            float p[4];
            shares<LPT>(v[k], p);
#pragma unroll
            for (int j = 0; j < 4; ++j) acc[j] += p[j];
        }
    }
#pragma unroll
    for (int j = 0; j < 4; ++j) lds.psum[grp][expert_of<LPT, VEC>(l, j)] = acc[j];
    __syncthreads();
    if (tid < E) {
        float p[4] = {0.f, 0.f, 0.f, 0.f};
        for (int g = 0; g < GROUPS; g += 4)
#pragma unroll
            for (int i = 0; i < 4; ++i) p[i] += lds.psum[g + i][tid];
        sum = (p[0] + p[1]) + (p[2] + p[3]);
        count = lds.cnt[tid];
    }
}

template <int LPT, bool VEC>
__global__ __launch_bounds__(64 * RUN_WAVES) void balance_runs_kernel(
    const float* __restrict__ s, const int32_t* __restrict__ idx, const int32_t* __restrict__ start, int n_seq, int T,
    int E, int K, int chunk, BalanceRun* __restrict__ rec, int32_t* __restrict__ chunk_n) {
    __shared__ RunLds<LPT> lds;
    const int tid = threadIdx.x;
    const int tb = blockIdx.x * chunk, te = min(T, tb + chunk);
    int all = 0;                                      // thread = expert: counts over the chunk's runs
    for (int q = seq_of<64>(start, n_seq, T, tb); q < n_seq; ++q) {
        const int rb = max(tb, seq_start_at(start, q, n_seq, T)), re = min(te, seq_start_at(start, q + 1, n_seq, T));
        if (rb >= te) break;
        if (rb >= re) {                               // an empty sequence has no record; nor have those behind it
            q = max(q, seq_of<64>(start, n_seq, T, rb) - 1);
            continue;
        }
        float p = 0.0f;
        int n = 0;
        run_sums<LPT, VEC>(s, idx, rb, re, E, K, lds, p, n);
        if (tid < E) {
            rec[blockIdx.x + q].p[tid] = p;
            rec[blockIdx.x + q].n[tid] = n;
            all += n;
        }
        __syncthreads();
    }
    if (tid < E) chunk_n[blockIdx.x * 256 + tid] = all;
}

// A sequence's count and loss from the sums over its L tokens: thread = expert, four
// waves.
__device__ __forceinline__ void finish_sequence(int e, float p, int n, int q, int L, int E, int K, float alpha,
                                                float (&wave_term)[4], float* loss, int32_t* seq_count) {
    if (e < E) seq_count[(int64_t)q * E + e] = n;
    const float len = (float)max(L, 1), f = (float)E * (float)n / ((float)K * len);
    const float term = wave_sum(f * (p / len));
    if ((e & 63) == 0) wave_term[e >> 6] = term;
    __syncthreads();
    if (e == 0) loss[q] = alpha * ((wave_term[0] + wave_term[1]) + (wave_term[2] + wave_term[3]));
}

// Small calls in one launch: a block goes through a whole sequence, and one counts over
// all of them.
template <int LPT, bool VEC>
__global__ __launch_bounds__(64 * RUN_WAVES) void balance_small_kernel(
    const float* __restrict__ s, const int32_t* __restrict__ idx, const int32_t* __restrict__ start, int n_seq, int T,
    int E, int K, float alpha, float* __restrict__ loss, int32_t* __restrict__ seq_count,
    int32_t* __restrict__ expert_count) {
    __shared__ RunLds<LPT> lds;
    __shared__ float wave_term[4];
    const int tid = threadIdx.x, q = blockIdx.x;
    if (q == n_seq) {
        if (tid < 256) lds.cnt[tid] = 0;
        __syncthreads();
        const int b = seq_start_at(start, 0, n_seq, T) * K, end = seq_start_at(start, n_seq, n_seq, T) * K;
        for (int i = b + tid; i < end; i += 64 * RUN_WAVES) {
            const int e = idx[i];
            if ((unsigned)e < (unsigned)E) atomicAdd(&lds.cnt[e], 1);
        }
        __syncthreads();
        if (tid < E) expert_count[tid] = lds.cnt[tid];
        return;
    }
    const int b = seq_start_at(start, q, n_seq, T), L = max(seq_start_at(start, q + 1, n_seq, T) - b, 0);
    float p = 0.0f;
    int n = 0;
    if (L > 0) run_sums<LPT, VEC>(s, idx, b, b + L, E, K, lds, p, n);
    if (tid < 256) finish_sequence(tid, p, n, q, L, E, K, alpha, wave_term, loss, seq_count);
}

// The sum of x(c) for c = c0 + part, c0 + part + 4, .. up to c1, in that order, 16 loads
// at a time.
template <typename V, typename Load>
__device__ __forceinline__ V every_fourth(int c0, int c1, int part, Load&& x) {
    V s = 0;
    for (int c = c0 + part; c <= c1; c += 64) {
        V v[16];
#pragma unroll
        for (int i = 0; i < 16; ++i) v[i] = x(min(c + 4 * i, c1));
#pragma unroll
        for (int i = 0; i < 16; ++i) s += c + 4 * i <= c1 ? v[i] : (V)0;
    }
    return s;
}

// One block per sequence, and one for the counts over all of them: thread = expert
// and one of four parts of the records (256 chunks in 4 sequences or 96: 6 us).
__global__ __launch_bounds__(1024) void balance_sum_kernel(const BalanceRun* __restrict__ rec,
                                                           const int32_t* __restrict__ chunk_n,
                                                           const int32_t* __restrict__ start, int n_seq, int T, int E,
                                                           int K, int chunk, float alpha, float* __restrict__ loss,
                                                           int32_t* __restrict__ seq_count,
                                                           int32_t* __restrict__ expert_count) {
    __shared__ float ps[4][256];
    __shared__ int ns[4][256];
    const int e = threadIdx.x & 255, part = threadIdx.x >> 8, q = blockIdx.x;
    if (q == n_seq) {
        ns[part][e] = e < E ? every_fourth<int>(0, (T + chunk - 1) / chunk - 1, part,
                                                [&](int c) { return chunk_n[c * 256 + e]; }) : 0;
        __syncthreads();
        if (part == 0 && e < E) expert_count[e] = (ns[0][e] + ns[1][e]) + (ns[2][e] + ns[3][e]);
        return;
    }
    const int b = seq_start_at(start, q, n_seq, T), L = max(seq_start_at(start, q + 1, n_seq, T) - b, 0);
    float p = 0.0f;
    int n = 0;
    if (L > 0 && e < E) {
        const int c0 = b / chunk, c1 = (b + L - 1) / chunk;
        p = every_fourth<float>(c0, c1, part, [&](int c) { return rec[c + q].p[e]; });
        n = every_fourth<int>(c0, c1, part, [&](int c) { return rec[c + q].n[e]; });
    }
    ps[part][e] = p;
    ns[part][e] = n;
    __syncthreads();
    if (part) return;
    p = (ps[0][e] + ps[1][e]) + (ps[2][e] + ps[3][e]);
    n = (ns[0][e] + ns[1][e]) + (ns[2][e] + ns[3][e]);
    __shared__ float wave_term[4];
    finish_sequence(e, p, n, q, L, E, K, alpha, wave_term, loss, seq_count);
}

// LPT lanes go through EACH consecutive tokens: their sequence is looked for once and
// followed from there, its f kept as long as it lasts.  Bound by HBM: 131072 x 256 in 96
// sequences 44 us (6.1 TB/s), 16384 x 256 in 4 10, four dependent reads long before a
// token's sequence is known (the starts held by lane where they are few: the same; 8
// tokens a lane: 46).  Tokens that would take 2^32 threads (2^28 of more than 64 experts,
// 2^30 of fewer) go in several launches, by block0 (stepping by the grid instead: 131072 x
// 256 3 us more).
//
// f is taken from the sequence's least one on, f_i = E (n_i - min n) / (K L), which leaves
// f_i - sum_j f_j p_j as it is (sum p = 1) and holds its error to what the f are apart: use
// that is even gives zeros.
constexpr int EACH = BALANCE_EACH;

template <int LPT, bool VEC, bool NT>
__global__ __launch_bounds__(256) void balance_backward_kernel(
    const float* __restrict__ s, const int32_t* __restrict__ seq_count, const int32_t* __restrict__ start, int n_seq,
    int T, int E, int K, float alpha, const float* __restrict__ dloss, const float* in, float* out, unsigned block0) {
    constexpr int GROUPS = 256 / LPT;
    typedef float v4f __attribute__((ext_vector_type(4)));
    const int l = threadIdx.x % LPT;
    const int64_t first = ((int64_t)(block0 + blockIdx.x) * GROUPS + threadIdx.x / LPT) * EACH;
    if (first >= T) return;                           // whole groups of lanes
    const int t0 = (int)first, te = min(T, t0 + EACH);
    int q = -1, qb = 0, qe = 0;                       // the sequence that holds the last token looked at, or none yet
    float f[4], coef = 0.0f;
    for (int tt = t0; tt < te; tt += AT_ONCE) {
        float v[AT_ONCE][4], g[AT_ONCE][4];
#pragma unroll
        for (int k = 0; k < AT_ONCE; ++k) {
            load_experts<LPT, VEC>(s + (int64_t)(tt + k) * E, l, E, tt + k < te, v[k]);
            load_experts<LPT, VEC>(in + (int64_t)(tt + k) * E, l, E, in && tt + k < te, g[k]);
        }
#pragma unroll
        for (int k = 0; k < AT_ONCE; ++k) {
            const int t = tt + k;
            if (t >= te) break;
            if (q < 0 || (t >= qe && q < n_seq)) {
                q = seq_of<LPT>(start, n_seq, T, t);
                qb = q < n_seq ? seq_start_at(start, q, n_seq, T) : T;
                qe = q < n_seq ? seq_start_at(start, q + 1, n_seq, T) : T;
                const float len = (float)max(qe - qb, 1), per = (float)E / ((float)K * len);
                coef = q < n_seq ? (dloss ? dloss[q] : 1.0f) * alpha / len : 0.0f;
                int n[4], least = INT_MAX;
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    const int e = expert_of<LPT, VEC>(l, j);
                    n[j] = q < n_seq && e < E ? seq_count[(int64_t)q * E + e] : INT_MAX;
                    least = min(least, n[j]);
                }
                least = lanes_min<LPT>(least);
#pragma unroll
                for (int j = 0; j < 4; ++j) f[j] = n[j] == INT_MAX ? 0.0f : per * (float)(n[j] - least);
            }
            float p[4], o[4];
            shares<LPT>(v[k], p);
            const float fp = token_sum<LPT>(__builtin_fmaf(f[3], p[3], f[2] * p[2]) + __builtin_fmaf(f[1], p[1], f[0] * p[0]));
            const bool inside = t >= qb;              // qb = T behind the last sequence
#pragma unroll
            for (int j = 0; j < 4; ++j)
                o[j] = inside ? __builtin_fmaf(coef * p[j] * (1.0f - v[k][j]), f[j] - fp, g[k][j]) : g[k][j];
            float* const row = out + (int64_t)t * E;
            if constexpr (VEC) {
                if (4 * l < E) put<NT>(reinterpret_cast<v4f*>(row + 4 * l), v4f{o[0], o[1], o[2], o[3]});
            } else {
#pragma unroll
                for (int j = 0; j < 4; ++j)
                    if (l + LPT * j < E) put<NT>(row + l + LPT * j, o[j]);
            }
        }
    }
}

int balance_chunk(int64_t T) {
    const int64_t c = (T + RUN_CHUNKS - 1) / RUN_CHUNKS;
    return (int)(c < RUN_LEAST ? RUN_LEAST : c);
}

}  // namespace

// One launch, or two: a block takes 16 tokens at a time (64 of up to 64 experts), 16 rounds
// of which take as long as the second launch; the starts are not known here, so the
// longest sequence is taken for all of a few tokens, or for twice the mean of up to four
// times as many (1024 x 256 in one of many sequences costs 24 for 8.5).  Kernels, us, one /
// two: 300 x 61 in 7 sequences 3.7 / 8.5, 1024 x 64 in one 7.8 / 7.8, 2048 x 64 in one 13.0
// / 7.9 and in 8 4.4 / 8.0, 512 x 256 in one 13.5 / 8.4, in 4 5.3 / 7.6 and in 512 4.2 /
// 89, 1024 x 256 in 64 3.8 / 12.5, 2048 x 256 in 4 13.6 / 8.7.  Past the limit many short
// sequences, which a block goes through one after the other, cost most: 1000 x 256 in 512
// 4.6, 1100 46, 3000 in 500 24, 4097 in as many 105.
bool small_call(int64_t T, int n_seq, int E) {
    const int64_t few = E > 64 ? 256 : 1024;
    return T <= few || (T <= 4 * few && T <= n_seq * (few / 2));
}

size_t balance_loss_ws_bytes(int64_t T, int n_seq) {
    if (small_call(T, n_seq, 256)) return 16;         // whatever E: small with 256 experts is small with fewer
    const int64_t chunk = balance_chunk(T);
    const int64_t chunks = (T + chunk - 1) / chunk;
    return (size_t)(chunks + n_seq) * sizeof(BalanceRun) + (size_t)chunks * 256 * sizeof(int32_t);
}

hipError_t launch_balance_loss(const float* s, const int32_t* idx, const int32_t* start, int n_seq, int64_t T, int E,
                               int K, float alpha, float* loss, int32_t* seq_count, int32_t* expert_count, void* ws,
                               hipStream_t st) {
    if (small_call(T, n_seq, E)) {
        const auto small = E > 64 ? E % 4 ? balance_small_kernel<64, false> : balance_small_kernel<64, true>
                                  : E % 4 ? balance_small_kernel<16, false> : balance_small_kernel<16, true>;
        hipLaunchKernelGGL(small, dim3(n_seq + (expert_count ? 1 : 0)), dim3(64 * RUN_WAVES), 0, st, s, idx, start, n_seq,
                           (int)T, E, K, alpha, loss, seq_count, expert_count);
        return hipGetLastError();
    }
    BalanceRun* rec = static_cast<BalanceRun*>(ws);
    const int chunk = balance_chunk(T), chunks = (int)((T + chunk - 1) / chunk);
    int32_t* chunk_n = reinterpret_cast<int32_t*>(rec + chunks + n_seq);
    const auto runs = E > 64 ? E % 4 ? balance_runs_kernel<64, false> : balance_runs_kernel<64, true>
                             : E % 4 ? balance_runs_kernel<16, false> : balance_runs_kernel<16, true>;
    hipLaunchKernelGGL(runs, dim3(chunks), dim3(64 * RUN_WAVES), 0, st, s, idx, start, n_seq, (int)T, E, K, chunk, rec,
                       chunk_n);
    hipLaunchKernelGGL(balance_sum_kernel, dim3(n_seq + (expert_count ? 1 : 0)), dim3(1024), 0, st, rec, chunk_n, start,
                       n_seq, (int)T, E, K, chunk, alpha, loss, seq_count, expert_count);
    return hipGetLastError();
}

hipError_t launch_balance_loss_backward(const float* s, const int32_t* seq_count, const int32_t* start, int n_seq,
                                        int64_t T, int E, int K, float alpha, const float* dloss, const float* in,
                                        float* out, hipStream_t st) {
    const bool nt = streamed(T * E * 4);
    const auto kernel = E > 64 ? E % 4 ? nt ? balance_backward_kernel<64, false, true> : balance_backward_kernel<64, false, false>
                                       : nt ? balance_backward_kernel<64, true, true> : balance_backward_kernel<64, true, false>
                               : E % 4 ? nt ? balance_backward_kernel<16, false, true> : balance_backward_kernel<16, false, false>
                                       : nt ? balance_backward_kernel<16, true, true> : balance_backward_kernel<16, true, false>;
    for (int64_t from = 0; from < T; from += balance_backward_tokens(E)) {
        hipLaunchKernelGGL(kernel, dim3(balance_backward_blocks(T - from, E)), dim3(256), 0, st, s, seq_count, start, n_seq,
                           (int)T, E, K, alpha, dloss, in, out, (unsigned)(from / balance_block_tokens(E)));
        const hipError_t e = hipGetLastError();
        if (e != hipSuccess) return e;
    }
    return hipSuccess;
}

size_t seq_balance_ws_bytes(int64_t n_seq, int L) {
    const int64_t nchunk = (L + BAL_CHUNK - 1) / BAL_CHUNK;
    return (size_t)(n_seq * nchunk) * sizeof(BalancePart);
}

hipError_t launch_seq_balance_loss(const float* s, const int32_t* idx, int64_t n_seq, int E, int K,
                                   int L, float alpha, float* loss, void* ws, hipStream_t st) {
    const int nchunk = (L + BAL_CHUNK - 1) / BAL_CHUNK;
    BalancePart* part = static_cast<BalancePart*>(ws);
    hipLaunchKernelGGL(seq_balance_partial_kernel, dim3((unsigned)(n_seq * nchunk)), dim3(64 * BAL_WAVES), 0,
                       st, s, idx, E, K, L, nchunk, part);
    hipLaunchKernelGGL(seq_balance_final_kernel, dim3((unsigned)n_seq), dim3(256), 0, st, part, E, K, L,
                       nchunk, alpha, loss);
    return hipGetLastError();
}

}  // namespace moe
