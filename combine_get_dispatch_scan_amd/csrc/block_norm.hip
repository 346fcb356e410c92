// The norms before and after a block with its gate and residual scales, on gfx950:
//   z  = y * rz,  rz = 1 / sqrt(mean y^2 + eps)      (or z = y)
//   x' = a x + fy gt z,  fy = b * channel gate * (o + y_weight),  gt = token gate
//   h  = x' r (o + weight),  r = 1 / sqrt(mean x'^2 + eps),  as bf16 and as FP8 rows
// and their gradients.  A team of lanes (a wave, or a workgroup of up to 16) holds a
// row in registers, so every value is read and written once; means are fp32 sums
// over the lanes.  All arithmetic is fp32, and every output is rounded once, by gfx950's
// converter: a NaN of any bits stays one.
//
// Memory bounds both: 16384 x 7168 in bf16 with y's norm, weights, a token gate and 8-bit
// rows takes 186 us forward, 5.7 TB/s (a copy of 1 GiB: 5.1), and 289 us backward, 4.9 TB/s.
// To keep it busy a team fetches its next row before it computes the one it has, and
// parameters are widened after all of them are on their way (with the wide loads of the
// second launch: 298 us, 373 without).  One row takes 4.3 us, of which the launch is most.
#include "block_launch.h"
#include "mfma.h"
#include "quant16.h"

namespace moe_ep {

constexpr int kTeamWaves = 16;               // waves of a row, at most
constexpr int64_t kSmallBytes = (int64_t)16 << 20, kLargeBytes = (int64_t)256 << 20;

template <int CTRL>
__device__ __forceinline__ float dpp_f(float v)
{
    return __int_as_float(__builtin_amdgcn_mov_dpp(__float_as_int(v), CTRL, 0xF, 0xF, true));
}

// Sum over a wave's lanes, the same in all of them: lane ^ 1, lane ^ 2, the other four
// of eight, the other eight of sixteen, then the four sixteens.
__device__ __forceinline__ float wave_sum(float v)
{
    v += dpp_f<0xB1>(v);
    v += dpp_f<0x4E>(v);
    v += dpp_f<0x141>(v);
    v += dpp_f<0x140>(v);
    return (readlane_f(v, 0) + readlane_f(v, 16)) + (readlane_f(v, 32) + readlane_f(v, 48));
}

__device__ __forceinline__ float max16(float m)
{
    m = max8(m);
    return fmaxf(m, dpp_f<0x140>(m));
}

// Sums over the team.  A workgroup's waves meet in LDS, in slots that are used in turn:
// a slot is written again only after the barrier of the sum in between.
template <bool WAVE, int N>
struct TeamSum {
    float (*slots)[kTeamWaves][N];
    int turn;

    __device__ __forceinline__ void operator()(float (&v)[N])
    {
#pragma unroll
        for (int i = 0; i < N; ++i)
            v[i] = wave_sum(v[i]);
        if (WAVE)
            return;
        const int wave = threadIdx.x / kWave, waves = blockDim.x / kWave;
        if (threadIdx.x % kWave == 0)
#pragma unroll
            for (int i = 0; i < N; ++i)
                slots[turn][wave][i] = v[i];
        __syncthreads();
#pragma unroll
        for (int i = 0; i < N; ++i)
            v[i] = slots[turn][0][i];
        for (int w = 1; w < waves; ++w)
#pragma unroll
            for (int i = 0; i < N; ++i)
                v[i] += slots[turn][w][i];
        turn ^= 1;
    }
};

// A row's mean square is sum((v * part) * v) * rest: part the largest power of two that is at most 1 / width, part * rest
// = 1 / width.  The sum then stays in fp32's range wherever the mean does (the sum of the squares themselves left it from
// values of 2^56.5 on at the largest width).  A power of two moves no rounding; only terms below 2^-126, which eps drowns,
// lose bits.
struct MeanSquare {
    float part, rest;

    __device__ __forceinline__ explicit MeanSquare(int width)
    {
        const int k = 32 - __clz(width - 1);              // 2^k: width, or the next power of two above it
        part = __uint_as_float((uint32_t)(127 - k) << 23);
        rest = 1.0f / (float)width * __uint_as_float((uint32_t)(127 + k) << 23);
    }
    __device__ __forceinline__ float add(float v, float sum) const { return __builtin_fmaf(v * part, v, sum); }
};

// Eight channels of a vector of parameters as they lie in memory (fp32, or bf16 twice).
// Loading and widening are apart, so that all loads are on their way before one is waited for.
struct RawParam8 {
    u32x4 d[2] = {u32x4{0u, 0u, 0u, 0u}, u32x4{0u, 0u, 0u, 0u}};

    __device__ __forceinline__ void load(const void* p, bool f32, int vec)
    {
        const char* q = static_cast<const char*>(p) + (size_t)vec * (f32 ? 32 : 16);
        d[0] = load16_hint<false>(q);
        d[1] = load16_hint<false>(q + (f32 ? 16 : 0));
    }
    __device__ __forceinline__ float get(bool f32, int j) const
    {
        const float wide = __uint_as_float(d[j >> 2][j & 3]);
        const float narrow = (j & 1) ? bf16_hi(d[0][j >> 1]) : bf16_lo(d[0][j >> 1]);
        return f32 ? wide : narrow;
    }
};

__device__ __forceinline__ float load_param(const void* p, bool f32, int i)
{
    if (f32)
        return static_cast<const float*>(p)[i];
    return __uint_as_float((uint32_t)static_cast<const uint16_t*>(p)[i] << 16);
}

__device__ __forceinline__ void store_param(void* p, bool f32, int i, float v)
{
    if (f32)
        static_cast<float*>(p)[i] = v;
    else
        static_cast<uint16_t*>(p)[i] = (uint16_t)pack2_bf16(v, v);
}

// The parameters of eight channels, and what they make up: y's factor and the norm's.
struct Factors8 {
    RawParam8 yw, gate, w;

    __device__ __forceinline__ void load_y(const ep_block_norm_t& a, int vec)
    {
        if (a.y_weight)
            yw.load(a.y_weight, a.weights_f32, vec);
        if (a.gate_kind == EP_GATE_CHANNEL)
            gate.load(a.gate, a.gate_f32, vec);
    }
    __device__ __forceinline__ void load_w(const ep_block_norm_t& a, int vec)
    {
        if (a.weight)
            w.load(a.weight, a.weights_f32, vec);
    }
    __device__ __forceinline__ void get_y(const ep_block_norm_t& a, float (&fy)[8]) const
    {
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            fy[j] = a.y_weight ? a.y_scale * (a.weight_offset + yw.get(a.weights_f32, j)) : a.y_scale;
            if (a.gate_kind == EP_GATE_CHANNEL)
                fy[j] *= gate.get(a.gate_f32, j);
        }
    }
    __device__ __forceinline__ void get_w(const ep_block_norm_t& a, float (&fw)[8]) const
    {
#pragma unroll
        for (int j = 0; j < 8; ++j)
            fw[j] = a.weight ? a.weight_offset + w.get(a.weights_f32, j) : 1.0f;
    }
};

// A lane's factors: kept in registers, or, in rows wider than 8192 (up to 1024 threads,
// 128 registers each), read again from memory at each use.
template <int V, bool KEEP>
struct Factors {
    float y[KEEP ? V : 1][8], w[KEEP ? V : 1][8];

    __device__ __forceinline__ void keep(const ep_block_norm_t& a, const Factors8 (&f)[V])
    {
#pragma unroll
        for (int i = 0; i < (KEEP ? V : 0); ++i) {
            f[i].get_y(a, y[i]);
            f[i].get_w(a, w[i]);
        }
    }
    __device__ __forceinline__ void get_y(const ep_block_norm_t& a, int i, int vec, bool on, float (&o)[8]) const
    {
        if (KEEP) {
#pragma unroll
            for (int j = 0; j < 8; ++j)
                o[j] = y[KEEP ? i : 0][j];
        } else {
            Factors8 f;
            if (on)
                f.load_y(a, vec);
            f.get_y(a, o);
        }
    }
    __device__ __forceinline__ void get_w(const ep_block_norm_t& a, int i, int vec, bool on, float (&o)[8]) const
    {
        if (KEEP) {
#pragma unroll
            for (int j = 0; j < 8; ++j)
                o[j] = w[KEEP ? i : 0][j];
        } else {
            Factors8 f;
            if (on)
                f.load_w(a, vec);
            f.get_w(a, o);
        }
    }
};

// Eight values of a row as they lie in memory: bf16 or fp32.
template <bool F32>
struct Raw8 {
    u32x4 d[F32 ? 2 : 1];

    __device__ __forceinline__ void zero()
    {
#pragma unroll
        for (int i = 0; i < (F32 ? 2 : 1); ++i)
            d[i] = u32x4{0u, 0u, 0u, 0u};
    }
    __device__ __forceinline__ void load(const void* p, size_t at)
    {
        const char* q = static_cast<const char*>(p) + at * (F32 ? 4 : 2);
#pragma unroll
        for (int i = 0; i < (F32 ? 2 : 1); ++i)
            d[i] = load16_hint<false>(q + 16 * i);
    }
    __device__ __forceinline__ float get(int j) const
    {
        if (F32)
            return __uint_as_float(d[F32 ? j >> 2 : 0][j & 3]);
        return (j & 1) ? bf16_hi(d[0][j >> 1]) : bf16_lo(d[0][j >> 1]);
    }
    template <bool NT = false>
    static __device__ __forceinline__ void store(void* p, size_t at, const float (&v)[8])
    {
        char* q = static_cast<char*>(p) + at * (F32 ? 4 : 2);
        if (F32) {
#pragma unroll
            for (int i = 0; i < 2; ++i)
                store16_hint<NT>(q + 16 * i, u32x4{__float_as_uint(v[4 * i]), __float_as_uint(v[4 * i + 1]),
                                                      __float_as_uint(v[4 * i + 2]), __float_as_uint(v[4 * i + 3])});
        } else {
            u32x4 o;
#pragma unroll
            for (int j = 0; j < 4; ++j)
                o[j] = pack2_bf16(v[2 * j], v[2 * j + 1]);
            store16_hint<NT>(q, o);
        }
    }
};

template <bool WAVE, int V, bool F32, int THREADS, bool NT>
__global__ __launch_bounds__(THREADS) void block_norm_kernel(BlockNormLaunch L)
{
    __shared__ float slots[2][kTeamWaves][1];
    const ep_block_norm_t& a = L.in;
    const int lane = WAVE ? threadIdx.x % kWave : threadIdx.x, lanes = WAVE ? kWave : blockDim.x;
    const int H = a.width, vecs = H / 8;
    const int teams = WAVE ? gridDim.x * (THREADS / kWave) : gridDim.x;
    const int first = WAVE ? blockIdx.x * (THREADS / kWave) + threadIdx.x / kWave : blockIdx.x;
    const MeanSquare square(H);
    TeamSum<WAVE, 1> sum{slots, 0};
    constexpr bool KEEP = THREADS <= 512;
    bool on[V];
    Factors8 f[KEEP ? V : 1];
    Factors<V, KEEP> factors;
    Raw8<F32> nx[V];
    Raw8<false> ny[V];
    // a row on its way while the one before it is computed: y from its start, x from its second half on (16384 x 7168
    // 186 us, 8192 x 4096 50; both from the start 198 and 51, both from the second half 191 and 59)
    const auto fetch_y = [&](int64_t row) {
#pragma unroll
        for (int i = 0; i < V; ++i)
            if (on[i] && a.y)
                ny[i].load(a.y, row * a.y_ld + (lane + i * lanes) * 8);
    };
    const auto fetch_x = [&](int64_t row) {
#pragma unroll
        for (int i = 0; i < V; ++i)
            if (on[i])
                nx[i].load(a.x, row * a.x_ld + (lane + i * lanes) * 8);
    };
    const auto fetch = [&](int64_t row) {
#pragma unroll
        for (int i = 0; i < V; ++i)
            if (on[i]) {
                const int c = (lane + i * lanes) * 8;
                nx[i].load(a.x, row * a.x_ld + c);
                if (a.y)
                    ny[i].load(a.y, row * a.y_ld + c);
            }
    };
#pragma unroll
    for (int i = 0; i < V; ++i) {
        on[i] = lane + i * lanes < vecs;
        nx[i].zero();
        ny[i].zero();
        if (KEEP && on[i]) {
            f[KEEP ? i : 0].load_y(a, lane + i * lanes);
            f[KEEP ? i : 0].load_w(a, lane + i * lanes);
        }
    }
    if (KEEP && first < a.num_rows)
        fetch(first);
    if constexpr (KEEP)
        factors.keep(a, f);
    for (int64_t row = first; row < a.num_rows; row += teams) {
        if (!KEEP)
            fetch(row);
        Raw8<F32> x[V];
        Raw8<false> y[V];
#pragma unroll
        for (int i = 0; i < V; ++i) {
            x[i] = nx[i];
            y[i] = ny[i];
        }
        if (KEEP && row + teams < a.num_rows)
            fetch_y(row + teams);
        float v[V][8];
        float ss[1] = {0.0f};
        if (a.y) {
            float cy = 1.0f;
            if (a.y_norm) {
#pragma unroll
                for (int i = 0; i < V; ++i)
#pragma unroll
                    for (int j = 0; j < 8; ++j)
                        ss[0] = square.add(y[i].get(j), ss[0]);
                sum(ss);
                cy = __builtin_amdgcn_rsqf(ss[0] * square.rest + a.eps);
            }
            if (a.gate_kind == EP_GATE_TOKEN)
                cy *= load_param(a.gate, a.gate_f32, (int)row);
#pragma unroll
            for (int i = 0; i < V; ++i) {
                float fy[8];
                factors.get_y(a, i, lane + i * lanes, on[i], fy);
#pragma unroll
                for (int j = 0; j < 8; ++j)
                    v[i][j] = __builtin_fmaf(a.residual_scale, x[i].get(j), y[i].get(j) * cy * fy[j]);
                if (L.xo && on[i])
                    Raw8<F32>::template store<NT>(L.xo, row * H + (lane + i * lanes) * 8, v[i]);
            }
        } else {
#pragma unroll
            for (int i = 0; i < V; ++i)
#pragma unroll
                for (int j = 0; j < 8; ++j)
                    v[i][j] = x[i].get(j);
        }
        if (KEEP && row + teams < a.num_rows)
            fetch_x(row + teams);
        if (!a.norm)
            continue;
        ss[0] = 0.0f;
#pragma unroll
        for (int i = 0; i < V; ++i)
#pragma unroll
            for (int j = 0; j < 8; ++j)
                ss[0] = square.add(v[i][j], ss[0]);
        sum(ss);
        const float r = __builtin_amdgcn_rsqf(ss[0] * square.rest + a.eps);
#pragma unroll
        for (int i = 0; i < V; ++i) {
            const int vec = lane + i * lanes;
            float fw[8];
            factors.get_w(a, i, vec, on[i], fw);
#pragma unroll
            for (int j = 0; j < 8; ++j)
                v[i][j] = v[i][j] * r * fw[j];
            if (L.h && on[i])
                Raw8<false>::template store<NT>(L.h, row * H + vec * 8, v[i]);
            if (L.codes) {
                // sixteen lanes hold a block of 128 (all of them on, or none)
                float m = 0.0f;
#pragma unroll
                for (int j = 0; j < 8; ++j)
                    m = fmaxf(m, fabsf(v[i][j]));
                const float top = fmaxf(max16(m), 0x1p-64f);
                const float k = 448.0f / top;
                uint32_t q[2];
#pragma unroll
                for (int j = 0; j < 2; ++j) {
                    q[j] = e4m3fn_pair<false>(v[i][4 * j] * k, v[i][4 * j + 1] * k, 0u);
                    q[j] = e4m3fn_pair<true>(v[i][4 * j + 2] * k, v[i][4 * j + 3] * k, q[j]);
                }
                if (on[i]) {
                    *reinterpret_cast<uint2*>(L.codes + row * H + vec * 8) = uint2{q[0], q[1]};
                    if ((vec & 15) == 0)
                        L.scales[row * (H / kQBlock) + vec / 16] = top / 448.0f;
                }
            }
        }
    }
}

// Backward.  Both factors of the row are computed again from x and y, so nothing but
// the inputs is kept between the passes:
//   d = gh (o + weight),  g = gx + r (d - x' r * mean(d x' r)),   dx = a g
//   s = sum over channels of g fy z  (the token gate's gradient)
//   dy = rz gt (g fy - z s / width)   (without y's norm: gt g fy)
//   dweight = sum over rows of gh x' r;  S = sum over rows of gt g z, from which
//   dy_weight = b * channel gate * S and the channel gate's gradient b (o + y_weight) S
// The sums over rows stay in the registers of the workgroups, which take rows in a fixed
// order, and are added by a second launch.  In rows of 8200 to 16384 they lie in LDS: 4096 x
// 16384 325 us, 356 with registers; the row and its factors still spill some 30 to 50 of 128
// registers there, and 300 to 360 in wider rows, whose sums are in registers again.  Stores go through the caches, unlike
// forward ones: with readers of dx and dy behind them that is as fast or faster at every
// size (8192 x 4096: 121 us, 134 around them).
template <bool WAVE, int V, bool F32, int THREADS>
__global__ __launch_bounds__(THREADS) void block_norm_backward_kernel(BlockNormBackwardLaunch L)
{
    __shared__ float slots[2][kTeamWaves][2];
    // [2][width].  WAVE: where the waves' sums meet; SUMS: where each lane has its own
    extern __shared__ __align__(16) float comb[];
    constexpr bool SUMS = THREADS == 1024 && V == 2;
    const ep_block_norm_t& a = L.in;
    const int lane = WAVE ? threadIdx.x % kWave : threadIdx.x, lanes = WAVE ? kWave : blockDim.x;
    const int H = a.width, vecs = H / 8;
    const int teams = WAVE ? gridDim.x * (THREADS / kWave) : gridDim.x;
    const int first = WAVE ? blockIdx.x * (THREADS / kWave) + threadIdx.x / kWave : blockIdx.x;
    const float inv = 1.0f / (float)H;
    const MeanSquare square(H);
    TeamSum<WAVE, 2> sum{slots, 0};
    constexpr bool KEEP = THREADS <= 512;
    bool on[V];
    Factors8 f[KEEP ? V : 1];
    Factors<V, KEEP> factors;
    Raw8<F32> nx[V], ngx[V];
    Raw8<false> ny[V], ngh[V];
    const auto fetch = [&](int64_t row) {
#pragma unroll
        for (int i = 0; i < V; ++i)
            if (on[i]) {
                const int c = (lane + i * lanes) * 8;
                nx[i].load(a.x, row * a.x_ld + c);
                if (a.y)
                    ny[i].load(a.y, row * a.y_ld + c);
                if (L.gx)
                    ngx[i].load(L.gx, row * H + c);
                if (L.gh)
                    ngh[i].load(L.gh, row * H + c);
            }
    };
#pragma unroll
    for (int i = 0; i < V; ++i) {
        on[i] = lane + i * lanes < vecs;
        nx[i].zero();
        ny[i].zero();
        ngx[i].zero();
        ngh[i].zero();
        if (KEEP && on[i]) {
            f[KEEP ? i : 0].load_y(a, lane + i * lanes);
            f[KEEP ? i : 0].load_w(a, lane + i * lanes);
        }
    }
    if (KEEP && first < a.num_rows)
        fetch(first);
    if constexpr (KEEP)
        factors.keep(a, f);
    float P[SUMS ? 1 : V][8], S[SUMS ? 1 : V][8];
#pragma unroll
    for (int i = 0; i < V; ++i)
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            P[SUMS ? 0 : i][j] = S[SUMS ? 0 : i][j] = 0.0f;
            if (SUMS && L.part && on[i])
                comb[(lane + i * lanes) * 8 + j] = comb[H + (lane + i * lanes) * 8 + j] = 0.0f;
        }
    // adds a b to a lane's sums of its vector i, P (which = 0) or S
    const auto add = [&](float (&kept)[SUMS ? 1 : V][8], int which, int i, const float (&a)[8], const float (&b)[8]) {
        if constexpr (SUMS) {
            if (L.part && on[i]) {
                float4* c = reinterpret_cast<float4*>(comb + which * H + (lane + i * lanes) * 8);
#pragma unroll
                for (int k = 0; k < 2; ++k) {
                    float4 v = c[k];
                    v.x = __builtin_fmaf(a[4 * k], b[4 * k], v.x);
                    v.y = __builtin_fmaf(a[4 * k + 1], b[4 * k + 1], v.y);
                    v.z = __builtin_fmaf(a[4 * k + 2], b[4 * k + 2], v.z);
                    v.w = __builtin_fmaf(a[4 * k + 3], b[4 * k + 3], v.w);
                    c[k] = v;
                }
            }
        } else {
#pragma unroll
            for (int j = 0; j < 8; ++j)
                kept[i][j] = __builtin_fmaf(a[j], b[j], kept[i][j]);
        }
    };
    for (int64_t row = first; row < a.num_rows; row += teams) {
        if (!KEEP)
            fetch(row);
        Raw8<F32> x[V], gx[V];
        Raw8<false> y[V], gh[V];
#pragma unroll
        for (int i = 0; i < V; ++i) {
            x[i] = nx[i];
            y[i] = ny[i];
            gx[i] = ngx[i];
            gh[i] = ngh[i];
        }
        if (KEEP && row + teams < a.num_rows)
            fetch(row + teams);
        float rz = 1.0f, gt = 1.0f;
        if (a.y_norm) {
            float ss[2] = {0.0f, 0.0f};
#pragma unroll
            for (int i = 0; i < V; ++i)
#pragma unroll
                for (int j = 0; j < 8; ++j)
                    ss[0] = square.add(y[i].get(j), ss[0]);
            sum(ss);
            rz = __builtin_amdgcn_rsqf(ss[0] * square.rest + a.eps);
        }
        if (a.gate_kind == EP_GATE_TOKEN)
            gt = load_param(a.gate, a.gate_f32, (int)row);
        float g[V][8];
#pragma unroll
        for (int i = 0; i < V; ++i)
#pragma unroll
            for (int j = 0; j < 8; ++j)
                g[i][j] = gx[i].get(j);
        if (L.gh) {
            float v[V][8];
            float ss[2] = {0.0f, 0.0f};
            const float cy = rz * gt;
#pragma unroll
            for (int i = 0; i < V; ++i) {
                float fy[8], fw[8];
                factors.get_y(a, i, lane + i * lanes, on[i], fy);
                factors.get_w(a, i, lane + i * lanes, on[i], fw);
#pragma unroll
                for (int j = 0; j < 8; ++j) {
                    v[i][j] = a.y ? __builtin_fmaf(a.residual_scale, x[i].get(j), y[i].get(j) * cy * fy[j])
                                  : x[i].get(j);
                    ss[0] = square.add(v[i][j], ss[0]);
                    ss[1] = __builtin_fmaf(gh[i].get(j) * fw[j], v[i][j], ss[1]);
                }
            }
            sum(ss);
            const float r = __builtin_amdgcn_rsqf(ss[0] * square.rest + a.eps);
            const float k = r * ss[1] * inv;
#pragma unroll
            for (int i = 0; i < V; ++i) {
                float fw[8], gv[8], xh[8];
                factors.get_w(a, i, lane + i * lanes, on[i], fw);
#pragma unroll
                for (int j = 0; j < 8; ++j) {
                    gv[j] = gh[i].get(j);
                    xh[j] = v[i][j] * r;
                    g[i][j] = __builtin_fmaf(r, gv[j] * fw[j] - xh[j] * k, g[i][j]);
                }
                add(P, 0, i, gv, xh);
            }
        }
        if (L.dx) {
#pragma unroll
            for (int i = 0; i < V; ++i)
                if (on[i]) {
                    float o[8];
#pragma unroll
                    for (int j = 0; j < 8; ++j)
                        o[j] = a.residual_scale * g[i][j];
                    Raw8<F32>::store(L.dx, row * H + (lane + i * lanes) * 8, o);
                }
        }
        if (!a.y)
            continue;
        float ss[2] = {0.0f, 0.0f};
#pragma unroll
        for (int i = 0; i < V; ++i) {
            float fy[8], gv[8], z[8];
            factors.get_y(a, i, lane + i * lanes, on[i], fy);
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                z[j] = y[i].get(j) * rz;
                gv[j] = gt * g[i][j];
                g[i][j] *= fy[j];
                ss[0] = __builtin_fmaf(g[i][j], z[j], ss[0]);
            }
            add(S, 1, i, gv, z);
        }
        if (a.y_norm || (L.dgate && a.gate_kind == EP_GATE_TOKEN))
            sum(ss);
        if (L.dgate && a.gate_kind == EP_GATE_TOKEN && lane == 0)
            store_param(L.dgate, a.gate_f32, (int)row, ss[0]);
        if (L.dy) {
            const float k = a.y_norm ? ss[0] * inv : 0.0f, c = rz * gt;
#pragma unroll
            for (int i = 0; i < V; ++i)
                if (on[i]) {
                    float o[8];
#pragma unroll
                    for (int j = 0; j < 8; ++j)
                        o[j] = c * (g[i][j] - y[i].get(j) * rz * k);
                    Raw8<false>::store(L.dy, row * H + (lane + i * lanes) * 8, o);
                }
        }
    }
    if (!L.part)
        return;
    float* part = L.part + (size_t)blockIdx.x * 2 * H;
    if (WAVE) {
        for (int w = 0; w < THREADS / kWave; ++w) {
            if ((int)threadIdx.x / kWave == w)
#pragma unroll
                for (int i = 0; i < V; ++i)
                    if (on[i])
#pragma unroll
                        for (int j = 0; j < 8; ++j) {
                            const int c = (lane + i * lanes) * 8 + j;
                            comb[c] = w ? comb[c] + P[i][j] : P[i][j];
                            comb[H + c] = w ? comb[H + c] + S[i][j] : S[i][j];
                        }
            __syncthreads();
        }
        for (int c = threadIdx.x; c < 2 * H; c += THREADS)
            part[c] = comb[c];
    } else if constexpr (SUMS) {
        __syncthreads();
        for (int c = threadIdx.x * 4; c < 2 * H; c += lanes * 4)
            *reinterpret_cast<float4*>(part + c) = *reinterpret_cast<const float4*>(comb + c);
    } else {
#pragma unroll
        for (int i = 0; i < V; ++i)
            if (on[i]) {
                Raw8<true>::store(part, (lane + i * lanes) * 8, P[i]);
                Raw8<true>::store(part, H + (lane + i * lanes) * 8, S[i]);
            }
    }
}

// The workgroups' sums: 64 columns a workgroup.  Sixteen lanes read a list entry's 64
// columns, so the workgroup takes 64 entries at a time; entry b goes to share b % 64, and
// the shares are added in their order.
constexpr int kReduceThreads = 1024, kShares = kReduceThreads / 16;

__global__ __launch_bounds__(kReduceThreads) void block_norm_reduce_kernel(BlockNormBackwardLaunch L, int blocks)
{
    __shared__ float got[kShares][kWave + 4];
    const ep_block_norm_t& a = L.in;
    const int H = a.width, which = blockIdx.y, c0 = blockIdx.x * kWave;
    if (which == 0 ? !L.dw : !(L.dyw || (L.dgate && a.gate_kind == EP_GATE_CHANNEL)))
        return;
    const int share = threadIdx.x / 16, at = (threadIdx.x % 16) * 4;
    float s[4] = {0.0f, 0.0f, 0.0f, 0.0f};
    if (c0 + at < H)                       // widths are multiples of eight: all four columns exist
        for (int b = share; b < blocks; b += kShares) {
            const u32x4 d = load16_hint<false>(L.part + ((size_t)b * 2 + which) * H + c0 + at);
#pragma unroll
            for (int j = 0; j < 4; ++j)
                s[j] += __uint_as_float(d[j]);
        }
#pragma unroll
    for (int j = 0; j < 4; ++j)
        got[share][at + j] = s[j];
    __syncthreads();
    // wave w adds shares 4 w .. 4 w + 3, the first wave the sixteen sums
    const int lane = threadIdx.x % kWave, wave = threadIdx.x / kWave, c = c0 + lane;
    float v = (got[4 * wave][lane] + got[4 * wave + 1][lane]) + (got[4 * wave + 2][lane] + got[4 * wave + 3][lane]);
    __syncthreads();
    got[wave][lane] = v;
    __syncthreads();
    if (wave || c >= H)
        return;
    v = 0.0f;
#pragma unroll
    for (int w = 0; w < kReduceThreads / kWave; ++w)
        v += got[w][lane];
    if (which == 0) {
        store_param(L.dw, a.weights_f32, c, v);
        return;
    }
    v *= a.y_scale;
    const bool channel = a.gate_kind == EP_GATE_CHANNEL;
    if (L.dyw)
        store_param(L.dyw, a.weights_f32, c, channel ? v * load_param(a.gate, a.gate_f32, c) : v);
    if (L.dgate && channel)
        store_param(L.dgate, a.gate_f32, c,
                    a.y_weight ? v * (a.weight_offset + load_param(a.y_weight, a.weights_f32, c)) : v);
}

// The team of a row: a wave with one or two vectors of eight a lane up to a width of
// 1024, else a workgroup with one vector up to 2048, two up to 16384, then four.  In us
// (16384 rows, bf16, both norms, token gate; forward, backward):
//   1024: wave 25, 51; workgroup 34, 63      2048: one vector 50, 86; two 53, 103
//   4096: two vectors 94, 163; one 100, 190
// From 8200 on a workgroup has up to 16 waves of 128 registers: factors are read again
// (L2) and the next row is not fetched ahead.  4096 x 16384 takes 134 us forward, 325
// backward (8 waves with four vectors each: 147, 388).  Registers are spilled to memory by the
// backward pass from 8200 on and by the forward pass beyond 16384 (21 and 37 of them): 2048 x
// 32768 takes 156 us forward, 897 backward, 0.9 TB/s.
struct Team {
    bool wave;
    int v, threads;
    int blocks(int rows, int most) const
    {
        const int64_t need = wave ? ((int64_t)rows + 3) / 4 : rows;
        return (int)(need < most ? need : most);
    }
    // Workgroups a CU takes at once.  Forward, in us: 16384 x 4096 94 with two, 127 with one, 101 with four; 16384 x 2048
    // 50 with four, 63 with two; 8191 x 2056 in fp32 (three waves) 43.6 with four, 44.1 with two, 34.9 and 35.9 with its
    // inputs in the Infinity Cache.  Backward (waves of 120 registers with one vector, 210 with two): 16384 x 2048 86
    // with three, 94 with two, 88 with four; 16384 x 1024 51 with two, 60 with four; 8192 x 4096 90 with two, 109 with
    // one; 4096 x 16384 325 with one, 345 with two
    int forward_blocks(int rows) const { return blocks(rows, kCus * (v == 1 || wave || threads <= 192 ? 4 : 2)); }
    int backward_blocks(int rows) const { return blocks(rows, kCus * (!wave && v == 1 ? 3 : threads <= 256 ? 2 : 1)); }
};

static Team team_of(int width)
{
    const int vecs = width / 8;
    if (vecs <= 128)
        return Team{true, vecs <= 64 ? 1 : 2, 256};
    const int v = vecs <= 256 ? 1 : vecs <= 2048 ? 2 : 4;
    return Team{false, v, ((vecs + v - 1) / v + kWave - 1) / kWave * kWave};
}

template <typename L, template <bool, int, bool, int> class K>
static hipError_t run_team(const char* name, const Team& t, const L& args, int blocks, size_t lds, hipStream_t stream)
{
    debug_launch(name, dim3(blocks), dim3(t.threads), lds);
    const bool f = args.in.x_f32;
    void (*kernel)(L);
    if (t.wave)
        kernel = t.v == 1 ? (f ? K<true, 1, true, 256>::get() : K<true, 1, false, 256>::get())
                          : (f ? K<true, 2, true, 256>::get() : K<true, 2, false, 256>::get());
    else if (t.v == 1)
        kernel = f ? K<false, 1, true, 256>::get() : K<false, 1, false, 256>::get();
    else if (t.v == 2 && t.threads <= 512)
        kernel = f ? K<false, 2, true, 512>::get() : K<false, 2, false, 512>::get();
    else if (t.v == 2)
        kernel = f ? K<false, 2, true, 1024>::get() : K<false, 2, false, 1024>::get();
    else
        kernel = f ? K<false, 4, true, 1024>::get() : K<false, 4, false, 1024>::get();
    kernel<<<blocks, t.threads, lds, stream>>>(args);
    return hipGetLastError();
}

template <bool WAVE, int V, bool F32, int THREADS>
struct Forward {
    static auto get() { return block_norm_kernel<WAVE, V, F32, THREADS, false>; }
};
template <bool WAVE, int V, bool F32, int THREADS>
struct ForwardAround {
    static auto get() { return block_norm_kernel<WAVE, V, F32, THREADS, true>; }
};
template <bool WAVE, int V, bool F32, int THREADS>
struct Backward {
    static auto get() { return block_norm_backward_kernel<WAVE, V, F32, THREADS>; }
};

hipError_t launch_block_norm(const BlockNormLaunch& L, hipStream_t stream)
{
    if (L.in.num_rows == 0)
        return hipSuccess;
    const Team t = team_of(L.in.width);
    const int blocks = t.forward_blocks(L.in.num_rows);
    // Outputs up to 16 MB are written through, which leaves less to write back at the kernel's end, and so are those that
    // the Infinity Cache cannot hold (256 MB).  In between, who reads them next finds them there.  With bf16 x' and h,
    // both read again by the next two calls, all of it in us, stores around the caches and through them:
    //   512 x 7168   26.7, 28.5     1024 x 4096  25.8, 27.3     1024 x 7168  33.1, 31.6
    //   8192 x 4096  97.0, 84.3     8192 x 7168   165, 158     16384 x 7168   309, 318
    const int64_t bytes = (int64_t)L.in.num_rows * L.in.width * ((L.xo ? L.in.x_f32 ? 4 : 2 : 0) + (L.h ? 2 : 0));
    if (bytes <= kSmallBytes || bytes > kLargeBytes)
        return run_team<BlockNormLaunch, ForwardAround>("block_norm", t, L, blocks, 0, stream);
    return run_team<BlockNormLaunch, Forward>("block_norm", t, L, blocks, 0, stream);
}

size_t block_norm_workspace(int rows, int width)
{
    const int blocks = team_of(width).backward_blocks(rows);
    return ((size_t)(blocks ? blocks : 1) * 2 * width * sizeof(float) + 255) / 256 * 256;
}

hipError_t launch_block_norm_backward(const BlockNormBackwardLaunch& L, hipStream_t stream)
{
    const Team t = team_of(L.in.width);
    const int blocks = t.backward_blocks(L.in.num_rows);
    if (blocks) {
        const bool sums = t.wave || (t.v == 2 && t.threads > 512);
        const size_t lds = sums && L.part ? (size_t)2 * L.in.width * sizeof(float) : 0;
        const hipError_t e = run_team<BlockNormBackwardLaunch, Backward>("block_norm_backward", t, L, blocks, lds, stream);
        if (e != hipSuccess)
            return e;
    }
    if (L.part) {
        const dim3 grid((L.in.width + kWave - 1) / kWave, 2);
        debug_launch("block_norm_reduce", grid, dim3(kReduceThreads), 0);
        block_norm_reduce_kernel<<<grid, kReduceThreads, 0, stream>>>(L, blocks);
    }
    return hipGetLastError();
}

}  // namespace moe_ep
