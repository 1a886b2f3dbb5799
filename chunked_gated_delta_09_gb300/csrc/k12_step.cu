// k12_step.cu -- the gated delta rule token by token on a pool of states (gdr_step).
//
// Each row v of a state S [V][K] goes by itself:
//     S' = S diag(exp g) ,  d = beta (v_v - S'_v . k) ,  S_v = S'_v + d k ,  o_v = scale S_v . q .
// A few tokens are taken so, in turn.  Over the L tokens that go together (up to 8) with G(s, t) the product of the decays after token s up to token t, this is
//     d_t = beta_t (v_t - S_0 . (G(0, t) k_t) - sum_{s < t} d_s A_ts) ,   A_ts = k_t . (G(s, t) k_s)
//     o_t = scale (S_0 . (G(0, t) q_t) + sum_{s <= t} d_s B_ts) ,         B_ts = q_t . (G(s, t) k_s)
//     S_L = S_0 G(0, L) + sum_s d_s (G(s, L) k_s) ,
// so all products of a row are with the state as it was read, none waits for the token before, and the vectors, A and B are
// formed once for all rows.  Decays are multiplied, never divided: a gate of -inf forgets and nothing else.
//
// A CTA has up to `rows` rows of one state, which come by asynchronous copies into shared memory while the vectors are formed.
// One token reads and writes each state once, 8 bytes for 8 operations: HBM bounds it (251 x 32 states of
// 128 x 128: 159 us, 6.68 TB/s).
#include "block_common.cuh"
#include "delta_step.h"
#include "tc_util.cuh"

namespace gdr {
namespace {

// What a CTA works on.
struct Place {
    int b, h, hk, first, rows, len = 0;
    float *state = nullptr;
    __device__ __forceinline__ explicit Place(const RuleStepParams &p) {
        b = blockIdx.x / p.Hv, h = blockIdx.x - b * p.Hv, hk = h / p.group;
        first = blockIdx.y * p.rows, rows = min(p.rows, p.V - first);
    }
    __device__ __forceinline__ void find(const RuleStepParams &p) {  // the state, and how many tokens count
        const int64_t slot = p.slots ? p.slots[b] : b;
        len = p.lengths ? min(max(p.lengths[b], 0), p.T) : p.T;
        if (slot < 0 || slot >= p.num_slots) len = 0;
        state = p.state + (len > 0 ? slot * p.state_stride : 0) + ((int64_t)h * p.V + first) * p.K;
    }
    template <typename T> __device__ __forceinline__ T *out(const RuleStepParams &p, int t) const {
        return static_cast<T *>(p.o) + (((int64_t)b * p.T + t) * p.Hv + h) * p.V + first;
    }
};

// ---------------------------------------------------------------- one token, or a few in turn
// A row lies on 8 lanes (16-byte pieces 8 lanes apart), 4 rows side by side in a warp and ROWS below each other; each piece
// is fetched by the thread that uses it, and rows stay in registers over the tokens.
constexpr int TURN_THREADS = 128, ROWS = 2, WARP_ROWS = 4 * ROWS;

// TM: tokens, at most.
template <int TM> struct alignas(16) TurnShared {
    float k[TM][128], q[TM][128], gamma[TM][128], v[TM][128];
    float4 kq[TM];  // k . q, a part from each warp
    float beta[TM];
};

__device__ __forceinline__ float sum_of(F2 a) {
    float x, y;
    a.get(x, y);
    return x + y;
}
__device__ __forceinline__ void load_piece(const float *p, F2 (&o)[2]) {
    const float4 x = *reinterpret_cast<const float4 *>(p);
    o[0] = F2(x.x, x.y), o[1] = F2(x.z, x.w);
}

// (rows and vectors are read 16 bytes at a time)
static_assert(sizeof(TurnShared<1>) % 16 == 0 && sizeof(TurnShared<3>) % 16 == 0 && sizeof(TurnShared<5>) % 16 == 0);

// NP: pieces of a row on each lane, K <= 32 NP.
template <typename T, int NP, int TM> __global__ void __launch_bounds__(TURN_THREADS) k12_turn(const RuleStepParams p) {
    extern __shared__ float4 raw[];
    TurnShared<TM> &sh = *reinterpret_cast<TurnShared<TM> *>(raw);
    float *tile = reinterpret_cast<float *>(&sh + 1);
    Place at(p);
    at.find(p);
    const int tid = threadIdx.x, sub = tid & 7, lead = (tid & 31) >> 3, col0 = sub * 4;
    if (p.o)
        for (int t = at.len; t < p.T; ++t)  // the tokens that do not count
            if (tid < at.rows) at.out<T>(p, t)[tid] = to_out_t<T>(0.f);
    if (at.len == 0) return;
    bool on[NP];
#pragma unroll
    for (int j = 0; j < NP; ++j) on[j] = j * 32 + col0 < p.K;
    const int row0 = (tid >> 5) * WARP_ROWS + lead;
    constexpr int NEXT = TURN_THREADS / 32 * WARP_ROWS;
    for (int row = row0; row < at.rows; row += NEXT)
#pragma unroll
        for (int r = 0; r < ROWS; ++r)
#pragma unroll
            for (int j = 0; j < NP; ++j)
                if (on[j] && row + 4 * r < at.rows) {
                    const int i = (row + 4 * r) * p.K + j * 32 + col0;
                    copy16(tile + i, at.state + i, true);
                }
    copies_issued();
    {
        // All of it is fetched before any of it is used; what is not there is fetched from the nearest place and dropped; no branch
        // between the tokens: each one's would wait for the last one's.
        const T *q = static_cast<const T *>(p.q), *k = static_cast<const T *>(p.k), *v = static_cast<const T *>(p.v);
        const int64_t token = (int64_t)at.b * p.T;
        const int c = min(tid, p.K - 1);
        const T *kp = k + token * p.k_ts + at.hk * p.k_hs + c, *qp = q ? q + token * p.q_ts + at.hk * p.q_hs + c : kp;
        const int64_t qs = q ? p.q_ts : p.k_ts;
        const T *vp = v + token * p.v_ts + at.h * p.v_hs + at.first + min(tid, at.rows - 1);
        const float *gp = p.g + token * p.g_ts + at.h * p.g_hs + (p.channel ? c : 0);
        T kr[TM], qr[TM], vr[TM];
        float ax[TM];
#pragma unroll
        for (int t = 0; t < TM; ++t) {
            const int64_t n = min(t, at.len - 1);
            kr[t] = kp[n * p.k_ts], qr[t] = qp[n * qs], vr[t] = vp[n * p.v_ts], ax[t] = gp[n * p.g_ts];
        }
        if (tid < at.len) sh.beta[tid] = load_scalar(p.beta, (token + tid) * p.beta_ts + at.h, p.beta_dtype);
#pragma unroll
        for (int t = 0; t < TM; ++t) {
            const float x = tid < p.K ? to_f32(kr[t]) : 0.f, y = tid < p.K ? to_f32(qr[t]) : 0.f;
            sh.k[t][tid] = x, sh.q[t][tid] = y, sh.gamma[t][tid] = expf(ax[t]), sh.v[t][tid] = to_f32(vr[t]);
            float kq = x * y;
#pragma unroll
            for (int m = 16; m >= 1; m /= 2) kq += __shfl_xor_sync(0xffffffffu, kq, m);
            if ((tid & 31) == 0) reinterpret_cast<float *>(&sh.kq[t])[tid >> 5] = kq;
        }
    }
    __syncthreads();
    copies_wait<0>();
    for (int row = row0; row - lead < at.rows; row += NEXT) {
        F2 s[ROWS][2 * NP];
#pragma unroll
        for (int r = 0; r < ROWS; ++r)
#pragma unroll
            for (int j = 0; j < NP; ++j) {
                F2 x[2] = {F2(0.f), F2(0.f)};
                if (on[j] && row + 4 * r < at.rows) load_piece(tile + (row + 4 * r) * p.K + j * 32 + col0, x);
                s[r][2 * j] = x[0], s[r][2 * j + 1] = x[1];
            }
#pragma unroll 1
        for (int t = 0; t < (TM == 1 ? 1 : at.len); ++t) {
            F2 x[ROWS], y[ROWS], kk[NP][2];  // products with k and with q
#pragma unroll
            for (int r = 0; r < ROWS; ++r) x[r] = y[r] = F2(0.f);
#pragma unroll
            for (int j = 0; j < NP; ++j) {
                F2 qq[2], g[2];
                load_piece(&sh.gamma[t][j * 32 + col0], g), load_piece(&sh.k[t][j * 32 + col0], kk[j]);
#pragma unroll
                for (int r = 0; r < ROWS; ++r) {
                    s[r][2 * j] = mul2(s[r][2 * j], g[0]), s[r][2 * j + 1] = mul2(s[r][2 * j + 1], g[1]);
                    x[r] = fma2(s[r][2 * j], kk[j][0], x[r]), x[r] = fma2(s[r][2 * j + 1], kk[j][1], x[r]);
                }
                if (!p.o) continue;
                load_piece(&sh.q[t][j * 32 + col0], qq);
#pragma unroll
                for (int r = 0; r < ROWS; ++r) y[r] = fma2(s[r][2 * j], qq[0], y[r]), y[r] = fma2(s[r][2 * j + 1], qq[1], y[r]);
            }
            float d[ROWS], o[ROWS];
#pragma unroll
            for (int r = 0; r < ROWS; ++r) d[r] = sum_of(x[r]), o[r] = sum_of(y[r]);
#pragma unroll
            for (int m = 1; m < 8; m *= 2)
#pragma unroll
                for (int r = 0; r < ROWS; ++r) {
                    d[r] += __shfl_xor_sync(0xffffffffu, d[r], m);
                    if (p.o) o[r] += __shfl_xor_sync(0xffffffffu, o[r], m);
                }
            const float4 kq = sh.kq[t];
#pragma unroll
            for (int r = 0; r < ROWS; ++r) {
                d[r] = sh.beta[t] * (sh.v[t][min(row + 4 * r, at.rows - 1)] - d[r]);
                if (p.o && sub == 0 && row + 4 * r < at.rows)
                    at.out<T>(p, t)[row + 4 * r] = to_out_t<T>(p.scale * fmaf(d[r], (kq.x + kq.y) + (kq.z + kq.w), o[r]));
#pragma unroll
                for (int j = 0; j < NP; ++j)
                    s[r][2 * j] = fma2(F2(d[r]), kk[j][0], s[r][2 * j]), s[r][2 * j + 1] = fma2(F2(d[r]), kk[j][1], s[r][2 * j + 1]);
            }
        }
        if (!p.update) continue;
#pragma unroll
        for (int r = 0; r < ROWS; ++r)
#pragma unroll
            for (int j = 0; j < NP; ++j)
                if (on[j] && row + 4 * r < at.rows) {
                    float4 n;
                    s[r][2 * j].get(n.x, n.y), s[r][2 * j + 1].get(n.z, n.w);
                    *reinterpret_cast<float4 *>(at.state + (row + 4 * r) * p.K + j * 32 + col0) = n;
                }
    }
}

// ---------------------------------------------------------------- tokens together
// The products of the rows with the 8 tokens' vectors, and those of d with u, are 16 x 8 x 8 products of the tensor cores, each
// operand split into the first 11 bits of its values and the rest (three products of parts: some 2^-21 off); the decayed state
// itself is not rounded to that, d u is added to it in fp32.  Warps have 16 rows; lane 4 g + c has columns 2 c and 2 c + 1
// of every eight in rows g and g + 8, and of tokens 2 c and 2 c + 1.
constexpr int FEW_TOKENS = 8;

struct Halves {  // the high and low parts of two neighbouring channels
    float hi0, hi1, lo0, lo1;
};
// CH: channels that there is room for; two threads for each.
template <int CH> struct alignas(16) FewShared {
    static constexpr int MAX_PAIRS = FEW_TOKENS * (FEW_TOKENS + 1) / 2, WARPS = CH / 32;  // of each half of the threads
    Halves k[FEW_TOKENS][CH / 2 + 4], q[FEW_TOKENS][CH / 2 + 4];  // G(0, t) k_t, G(0, t) q_t; rows apart by 64 bytes of banks
    float2 u[FEW_TOKENS][CH + 4];                                 // G(s, L) k_s, high and low parts; rows apart by 32 bytes of banks
    float gamma[CH];                                              // G(0, L)
    float v[FEW_TOKENS][128], beta[FEW_TOKENS];
    float a[FEW_TOKENS][FEW_TOKENS], b[FEW_TOKENS][FEW_TOKENS];   // beta_t A_ts and B_ts at [s][t]
    float part[2 * WARPS][MAX_PAIRS];
};
// Rows of the state in shared memory, 32 bytes of banks apart.
constexpr int FEW_PAD = 8;

__device__ __forceinline__ float high_part(float x) { return __uint_as_float(__float_as_uint(x) & 0xffffe000u); }
__device__ __forceinline__ void mma1688(float (&d)[4], const float (&a)[4], float b0, float b1) {
    asm volatile("mma.sync.aligned.m16n8k8.row.col.f32.tf32.tf32.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
                 : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
                 : "r"(__float_as_uint(a[0])), "r"(__float_as_uint(a[1])), "r"(__float_as_uint(a[2])), "r"(__float_as_uint(a[3])),
                   "r"(__float_as_uint(b0)), "r"(__float_as_uint(b1)));
}

// Sums over the warp of N values, at most 36, to to[0 .. N).
template <int N> __device__ __forceinline__ void warp_sums(const float (&x)[N], float *to) {
    const int lane = threadIdx.x & 31;
    if constexpr (N <= 16) {
        float y[16];
#pragma unroll
        for (int i = 0; i < 16; ++i) y[i] = i < N ? x[i] : 0.f;
        const float s = tc::warp_transpose_sum16(y);
        if (lane < N) to[lane] = s;
    } else {
        float y[32];
#pragma unroll
        for (int i = 0; i < 32; ++i) y[i] = i < N ? x[i] : 0.f;
        const float s = tc::warp_transpose_sum32(y);
        if (lane < N) to[lane] = s;
#pragma unroll
        for (int i = 32; i < N; ++i) {
            float z = x[i];
#pragma unroll
            for (int m = 16; m >= 1; m /= 2) z += __shfl_xor_sync(0xffffffffu, z, m);
            if (lane == 0) to[i] = z;
        }
    }
}

// LM: tokens that go together, at most.
template <typename T, int LM, int CH> __global__ void __launch_bounds__(2 * CH, 256 / CH) k12_few(const RuleStepParams p) {
    extern __shared__ float4 raw[];
    using Shared = FewShared<CH>;
    constexpr int FEW_THREADS = 2 * CH;
    Shared &sh = *reinterpret_cast<Shared *>(raw);
    float *tile = reinterpret_cast<float *>(&sh + 1);
    Place at(p);
    const int tid = threadIdx.x, lane = tid & 31, pitch = p.K + FEW_PAD;
    // A channel for two threads: the first has the keys, u and A, the second the queries and B; all of them have values.
    const int channel = tid & (CH - 1);
    const bool second = tid >= CH;
    constexpr int VALUES = (128 + FEW_THREADS - 1) / FEW_THREADS;
    T kr[LM], qr[LM], vr[VALUES][LM];
    float ax[LM], beta = 0.f;
    // The inputs of tokens t0 .. t0 + n, on their way while the state is found.  What is not there is fetched from the nearest place
    // and dropped; no branch between them: each token's would wait for the last one's.
    auto inputs = [&](int t0, int n) {
        const T *k = static_cast<const T *>(p.k), *q = static_cast<const T *>(p.q), *v = static_cast<const T *>(p.v);
        const int64_t token = (int64_t)at.b * p.T + t0;
        const int c = min(channel, p.K - 1);
        const T *kp = k + token * p.k_ts + at.hk * p.k_hs + c;
        const T *qp = second && q ? q + token * p.q_ts + at.hk * p.q_hs + c : kp;
        const int64_t qs = second && q ? p.q_ts : p.k_ts;
        const T *vp = v + token * p.v_ts + at.h * p.v_hs + at.first;
        const float *gp = p.g + token * p.g_ts + at.h * p.g_hs + (p.channel ? c : 0);
#pragma unroll
        for (int t = 0; t < LM; ++t) {
            const int64_t i = min(t, n - 1);
            kr[t] = kp[i * p.k_ts], qr[t] = qp[i * qs], ax[t] = gp[i * p.g_ts];
#pragma unroll
            for (int j = 0; j < VALUES; ++j) vr[j][t] = vp[i * p.v_ts + min(tid + j * FEW_THREADS, at.rows - 1)];
        }
        if (tid < n) beta = load_scalar(p.beta, (token + tid) * p.beta_ts + at.h, p.beta_dtype);
    };
    inputs(0, min(p.T, LM));
    at.find(p);
    if (p.o)
        for (int t = at.len; t < p.T; ++t)  // the tokens that do not count
            for (int row = tid; row < at.rows; row += FEW_THREADS) at.out<T>(p, t)[row] = to_out_t<T>(0.f);
    if (at.len == 0) return;
    for (int row = tid >> 3; row < at.rows; row += FEW_THREADS / 8)
        for (int c = (tid & 7) * 4; c < p.K; c += 32) copy16(tile + row * pitch + c, at.state + row * p.K + c, true);
    copies_issued();

    for (int t0 = 0; t0 < at.len; t0 += LM) {
        const int L = min(at.len - t0, LM);
        const bool last = t0 + LM >= at.len;
        {
            float kx[LM], ox[LM];
            if (tid < FEW_TOKENS) sh.beta[tid] = tid < L ? beta : 0.f;
#pragma unroll
            for (int t = 0; t < FEW_TOKENS; ++t)
#pragma unroll
                for (int i = 0; i < VALUES; ++i)
                    if (tid + i * FEW_THREADS < 128) sh.v[t][tid + i * FEW_THREADS] = t < LM && t < L ? to_f32(vr[i][t % LM]) : 0.f;
#pragma unroll
            for (int t = 0; t < LM; ++t) {
                const bool there = t < L && channel < p.K;
                kx[t] = there ? to_f32(kr[t]) : 0.f, ox[t] = there ? to_f32(qr[t]) : 0.f;
                ax[t] = t < L ? expf(ax[t]) : 1.f;
            }
            float g = 1.f;
            float *to = reinterpret_cast<float *>(second ? &sh.q[0][channel / 2] : &sh.k[0][channel / 2]) + (channel & 1);
            constexpr int NEXT = sizeof(sh.k[0]) / sizeof(float);
#pragma unroll
            for (int t = 0; t < FEW_TOKENS; ++t) {
                float x = 0.f;
                if (t < LM) {
                    g *= ax[t % LM];
                    x = g * (second ? ox[t % LM] : kx[t % LM]);
                }
                to[t * NEXT] = high_part(x), to[t * NEXT + 2] = x - high_part(x);
            }
            if (second) {
                float sums[LM * (LM + 1) / 2];
#pragma unroll
                for (int s = 0; s < LM; ++s) {
                    float w = kx[s];
#pragma unroll
                    for (int t = s; t < LM; ++t) {
                        if (t > s) w *= ax[t];
                        sums[t * (t + 1) / 2 + s] = ox[t] * w;
                    }
                }
                warp_sums(sums, sh.part[tid >> 5]);
            } else {
                sh.gamma[channel] = g;
                float sums[LM * (LM - 1) / 2];
#pragma unroll
                for (int s = 0; s < FEW_TOKENS; ++s) {
                    float w = 0.f;
                    if (s < LM) {
                        w = kx[s % LM];
#pragma unroll
                        for (int t = s + 1; t < LM; ++t) {
                            w *= ax[t];
                            sums[t * (t - 1) / 2 + s] = kx[t] * w;
                        }
                    }
                    sh.u[s][channel] = make_float2(high_part(w), w - high_part(w));  // (decays past L are 1)
                }
                warp_sums(sums, sh.part[tid >> 5]);
            }
        }
        __syncthreads();
        if (tid < FEW_TOKENS * FEW_TOKENS) {
            const int s = tid / FEW_TOKENS, t = tid % FEW_TOKENS;
            float a = 0.f, b = 0.f;
#pragma unroll
            for (int w = 0; w < Shared::WARPS; ++w) {
                if (s <= t && t < LM) b += sh.part[Shared::WARPS + w][t * (t + 1) / 2 + s];
                if (s < t && t < LM) a += sh.part[w][t * (t - 1) / 2 + s];
            }
            sh.a[s][t] = sh.beta[t] * a, sh.b[s][t] = b;
        }
        if (t0 == 0) copies_wait<0>();
        __syncthreads();

        const int g = lane >> 2, c = lane & 3;
        for (int row0 = (tid >> 5) * 16 + g; row0 - g < at.rows; row0 += FEW_THREADS / 32 * 16) {
            float *x0 = tile + row0 * pitch + 2 * c, *x1 = x0 + 8 * pitch;
            float sk3[3][4] = {}, sq3[3][4] = {};  // by the parts that were multiplied: sums of their own wait less
#pragma unroll 4
            for (int n = 0; n < p.K; n += 8) {
                const float2 y0 = *reinterpret_cast<const float2 *>(x0 + n), y1 = *reinterpret_cast<const float2 *>(x1 + n);
                const float y[4] = {y0.x, y1.x, y0.y, y1.y};
                float hi[4], lo[4];
#pragma unroll
                for (int i = 0; i < 4; ++i) hi[i] = high_part(y[i]), lo[i] = y[i] - hi[i];
                const Halves kk = sh.k[g][n / 2 + c], qq = sh.q[g][n / 2 + c];
                mma1688(sk3[0], hi, kk.hi0, kk.hi1), mma1688(sq3[0], hi, qq.hi0, qq.hi1);
                mma1688(sk3[1], lo, kk.hi0, kk.hi1), mma1688(sq3[1], lo, qq.hi0, qq.hi1);
                mma1688(sk3[2], hi, kk.lo0, kk.lo1), mma1688(sq3[2], hi, qq.lo0, qq.lo1);
            }
            float sk[4], sq[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) sk[i] = sk3[0][i] + (sk3[1][i] + sk3[2][i]), sq[i] = sq3[0][i] + (sq3[1][i] + sq3[2][i]);
            const int r0 = min(row0, at.rows - 1), r1 = min(row0 + 8, at.rows - 1);
            float d[2][2], ds[2][FEW_TOKENS];  // of rows g and g + 8: of the lane's tokens, and of all of them
#pragma unroll
            for (int j = 0; j < 2; ++j) {
                d[0][j] = sh.beta[2 * c + j] * (sh.v[2 * c + j][r0] - sk[j]);
                d[1][j] = sh.beta[2 * c + j] * (sh.v[2 * c + j][r1] - sk[2 + j]);
            }
#pragma unroll
            for (int t = 0; t < FEW_TOKENS; ++t) {
                if (t >= LM || t >= L) {
                    ds[0][t] = ds[1][t] = 0.f;
                    continue;
                }
                const float2 a = *reinterpret_cast<const float2 *>(&sh.a[t][2 * c]), b = *reinterpret_cast<const float2 *>(&sh.b[t][2 * c]);
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                    const float x = ds[i][t] = __shfl_sync(0xffffffffu, d[i][t & 1], (lane & ~3) | t >> 1);
                    // (above the diagonal a and b are 0: only what comes after token t is told by it)
                    if (2 * c > t) d[i][0] = fmaf(-x, a.x, d[i][0]);
                    if (2 * c + 1 > t) d[i][1] = fmaf(-x, a.y, d[i][1]);
                    if (2 * c >= t) sq[2 * i] = fmaf(x, b.x, sq[2 * i]);
                    if (2 * c + 1 >= t) sq[2 * i + 1] = fmaf(x, b.y, sq[2 * i + 1]);
                }
            }
            if (p.o)
#pragma unroll
                for (int j = 0; j < 2; ++j)
                    if (2 * c + j < L) {
                        T *o = at.out<T>(p, t0 + 2 * c + j);
                        if (row0 < at.rows) o[row0] = to_out_t<T>(p.scale * sq[j]);
                        if (row0 + 8 < at.rows) o[row0 + 8] = to_out_t<T>(p.scale * sq[2 + j]);
                    }
            if (!last || p.update) {
                float y[4], hi[4], lo[4];
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const float *x = &ds[i & 1][i >> 1 << 2];
                    y[i] = c & 2 ? (c & 1 ? x[3] : x[2]) : (c & 1 ? x[1] : x[0]);
                    hi[i] = high_part(y[i]), lo[i] = y[i] - hi[i];
                }
                float *to0 = last ? at.state + row0 * p.K + 2 * c : x0, *to1 = to0 + 8 * (last ? p.K : pitch);
#pragma unroll 4
                for (int n = 0; n < p.K; n += 8) {
                    const float2 u0 = sh.u[c][n + g], u1 = sh.u[c + 4][n + g], gamma = *reinterpret_cast<const float2 *>(&sh.gamma[n + 2 * c]);
                    float du[4] = {}, dv[4] = {}, dw[4] = {};
                    mma1688(du, hi, u0.x, u1.x), mma1688(dv, lo, u0.x, u1.x), mma1688(dw, hi, u0.y, u1.y);
#pragma unroll
                    for (int i = 0; i < 4; ++i) du[i] += dv[i] + dw[i];
                    const float2 s0 = *reinterpret_cast<const float2 *>(x0 + n), s1 = *reinterpret_cast<const float2 *>(x1 + n);
                    if (row0 < at.rows)
                        *reinterpret_cast<float2 *>(to0 + n) = make_float2(fmaf(gamma.x, s0.x, du[0]), fmaf(gamma.y, s0.y, du[1]));
                    if (row0 + 8 < at.rows)
                        *reinterpret_cast<float2 *>(to1 + n) = make_float2(fmaf(gamma.x, s1.x, du[2]), fmaf(gamma.y, s1.y, du[3]));
                }
            }
        }
        if (!last) {
            inputs(t0 + LM, min(p.T - t0 - LM, LM));
            __syncthreads();
        }
    }
}

template <typename T, int NP, int TM> cudaError_t turn_t(const RuleStepParams &p, cudaStream_t stream) {
    const cudaError_t e = smem_opt_in((const void *)k12_turn<T, NP, TM>, sizeof(TurnShared<TM>) + 64 * 128 * sizeof(float));
    if (e != cudaSuccess) return e;
    const dim3 grid((unsigned)(p.B * p.Hv), (unsigned)((p.V + p.rows - 1) / p.rows));
    k12_turn<T, NP, TM><<<grid, TURN_THREADS, sizeof(TurnShared<TM>) + (size_t)p.rows * p.K * sizeof(float), stream>>>(p);
    return cudaGetLastError();
}
template <typename T, int NP> cudaError_t turn_of(const RuleStepParams &p, cudaStream_t stream) {
    return p.T == 1 ? turn_t<T, NP, 1>(p, stream) : p.T <= 3 ? turn_t<T, NP, 3>(p, stream) : turn_t<T, NP, 5>(p, stream);
}
template <typename T, int LM, int CH> cudaError_t few_t(const RuleStepParams &p, cudaStream_t stream) {
    const cudaError_t e = smem_opt_in((const void *)k12_few<T, LM, CH>, sizeof(FewShared<CH>) + 128 * (CH + FEW_PAD) * sizeof(float));
    if (e != cudaSuccess) return e;
    const size_t smem = sizeof(FewShared<CH>) + (size_t)((p.rows + 15) / 16 * 16) * (p.K + FEW_PAD) * sizeof(float);
    k12_few<T, LM, CH><<<(unsigned)(p.B * p.Hv), 2 * CH, smem, stream>>>(p);
    return cudaGetLastError();
}
template <typename T, int CH> cudaError_t few_of(const RuleStepParams &p, cudaStream_t stream) {
    return p.T <= 3 ? few_t<T, 3, CH>(p, stream) : p.T <= 5 ? few_t<T, 5, CH>(p, stream) : few_t<T, 8, CH>(p, stream);
}
template <typename T> cudaError_t step_of(RuleStepParams p, cudaStream_t stream) {
    // Tokens in turn, or all products with the state as it was read.  us in turn and together, 256 x 32 states of 128 x 128, 64 x 64
    // and 32 x 32:
    //     states moved   2 tokens  167, 238   50, 72   27, 29        outputs alone   2 tokens  131, 134   43, 54   26, 25
    //                    4         238, 250   74, 78   38, 33                        3         164, 135   54, 54   30, 25
    //                    5         271, 252   84, 79   42, 33                        5         248, 150   80, 61   41, 29
    // So moved states go in turn up to 4 tokens where rows are long, and outputs alone up to 2; the fifth token, and the fourth of
    // states of 32 x 32, cost up to 27 % more in turn, but stay in fp32.  16 x 32 states of 128 x 128: 14 and 19 for 2 tokens
    // that move them, 20 and 20 for 4, 22 and 20 for 5.
    // In turn, 64 rows to a CTA (one token: 158 us, 160 with 128, 176 with 32; of 16 x 32 states 11.6, 14.6, 11.6); together, all
    // of them, since each CTA forms the vectors again.
    const bool turn = p.T <= (p.update ? 5 : 2);
    p.rows = turn && p.V > 64 ? 64 : p.V;
    if (turn) return p.K <= 32 ? turn_of<T, 1>(p, stream) : p.K <= 64 ? turn_of<T, 2>(p, stream) : turn_of<T, 4>(p, stream);
    return p.K <= 32 ? few_of<T, 32>(p, stream) : p.K <= 64 ? few_of<T, 64>(p, stream) : few_of<T, 128>(p, stream);
}

}  // namespace

cudaError_t launch_rule_step(const RuleStepParams &p, cudaStream_t stream) {
    if (p.dtype == F32) return step_of<float>(p, stream);
    if (p.dtype == BF16) return step_of<__nv_bfloat16>(p, stream);
    return step_of<__half>(p, stream);
}

}  // namespace gdr
