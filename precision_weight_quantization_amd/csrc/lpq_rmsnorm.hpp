// Root-mean-square norm with the residual's addition and MXFP8 output, and its
// backward pass.
//
// Part of lpq_kernels.hip, which includes each part once, in this order: one
// translation unit.
#pragma once

namespace {

// Forward, per row of N:
//   h = BF16(x + residual)                       (h = x without a residual)
//   r = 1 / sqrt(sum(h^2) / N + eps)             FP32
//   y = BF16(fl(fl(h * r) * gamma)), and the MXFP8 codes of y
// Backward, from g = dy * gamma and n = h * r:
//   dx     = BF16(r * (g - n * sum(g * n) / N) + dres)
//   dgamma = sum over the rows of dy * n         FP32
//
// Both read every array once, so HBM traffic is the floor, and work on a row out of
// registers between the reduction and the result.  G threads share a row, U vectors
// of 8 elements each: part of a wave for short rows (several rows per wave), one
// wave up to 4096 elements (the row's sum is then lane exchanges, without LDS or a
// barrier), a workgroup above.  The forward pass holds its rows without spilling.
// The gradients do up to 8192 elements (one wave a SIMD with 256 registers and the
// rest in accumulation registers from 2048 on); above, 1024 threads leave a lane 128
// registers: <1024, 2> (up to 16384) spills 8 of them, <1024, 4> (up to 32768) 112.
// Measured, with a residual, 168 MB (147 with MXFP8 output), buffers larger than
// the memory-side cache: 8192 x 2560 norm with MXFP8 output 28.8 us, 5.1 TB/s, with
// BF16 31.6; 2560 x 8192 28.7 and 30.0; 640 x 32768 32.0 and 32.4.  Gradients: 8192 x
// 2560 34.3 us without dgamma, 39.0 with (36.0 + 4.1 by themselves); 2560 x 8192 34.3
// and 40.8; 1280 x 16384 34.5 and 44.5; 640 x 32768 134 and 145, the spills.  98301 x
// 128 gradients (76 MB) 15.6 us, 4.8 TB/s, and 3.9 us for the sum of the partials.
// One row of 2560 takes 3.8 us, a launch and a few round trips to memory.
constexpr int kNormMaxN = 32768;

struct NormArgs {
    const uint16_t *x, *residual, *gamma;
    uint16_t *h, *y;
    float* rstd;
    uint8_t *q, *e;
    int64_t M;
    int32_t N;
    float eps;
};

struct NormGradArgs {
    const uint16_t *dy, *h, *gamma, *dres;
    const float* rstd;
    uint16_t* dx;
    float* part;         // [workgroups, N] partial sums of dgamma (NULL: no dgamma)
    int64_t M;
    int32_t N;
};

constexpr int norm_threads(int G) { return G > 256 ? G : 256; }

// Sum over the G threads of a row, the same bits in each of them: lane
// exchanges inside a wave, then the waves' sums through LDS in wave order.
// `slot` (0 or 1) alternates between calls so that one barrier is enough.
template <int G>
__device__ __forceinline__ float row_sum(float s, float (&lds)[2][16], int slot) {
#pragma unroll
    for (int k = 1; k < (G < 64 ? G : 64); k *= 2) s += __shfl_xor(s, k);
    if constexpr (G > 64) {
        if ((threadIdx.x & 63) == 0) lds[slot][threadIdx.x >> 6] = s;
        __syncthreads();
        s = lds[slot][0];
#pragma unroll
        for (int k = 1; k < G / 64; k++) s += lds[slot][k];
    }
    return s;
}

template <int G, int U>
__global__ __launch_bounds__(norm_threads(G)) void k_rmsnorm(NormArgs A) {
    constexpr int kRows = norm_threads(G) / G;
    __shared__ float lds[2][16];
    const int t = threadIdx.x % G;
    const int64_t row = (int64_t)blockIdx.x * kRows + threadIdx.x / G;
    const bool in_row = row < A.M;   // uniform over the row's threads
    const int64_t at = row * A.N;
    v4u h[U];
    float ss = 0.0f;
#pragma unroll
    for (int u = 0; u < U; u++) {
        const int c = (u * G + t) * 8;
        const bool in = in_row && c < A.N;
        h[u] = in ? load<kNTL>(reinterpret_cast<const v4u*>(A.x + at + c)) : v4u{};
    }
    // gamma's loads go out with the row's: a wave of few rows would wait for them after the sum
    v4u gm[U];
#pragma unroll
    for (int u = 0; u < U; u++) {
        const int c = (u * G + t) * 8;
        gm[u] = c < A.N ? load<false>(reinterpret_cast<const v4u*>(A.gamma + c)) : v4u{};
    }
    if (A.residual) {
        v4u r[U];
#pragma unroll
        for (int u = 0; u < U; u++) {
            const int c = (u * G + t) * 8;
            r[u] = in_row && c < A.N ? load<kNTL>(reinterpret_cast<const v4u*>(A.residual + at + c)) : v4u{};
        }
#pragma unroll
        for (int u = 0; u < U; u++) {
#pragma unroll
            for (int k = 0; k < 4; k++)
                h[u][k] = bf16x2(bf16_lo(h[u][k]) + bf16_lo(r[u][k]), bf16_hi(h[u][k]) + bf16_hi(r[u][k]));
        }
    }
#pragma unroll
    for (int u = 0; u < U; u++) {
        const int c = (u * G + t) * 8;
        if (A.h && in_row && c < A.N) store<kNTS>(reinterpret_cast<v4u*>(A.h + at + c), h[u]);
        const F8 f = widen8(h[u]);
#pragma unroll
        for (int k = 0; k < 8; k++) ss = __builtin_fmaf(f.x[k], f.x[k], ss);
    }
    ss = row_sum<G>(ss, lds, 0);
    const float r = 1.0f / __builtin_sqrtf(ss / (float)A.N + A.eps);
    if (A.rstd && in_row && t == 0) A.rstd[row] = r;
#pragma unroll
    for (int u = 0; u < U; u++) {
        const int c = (u * G + t) * 8;
        const bool in = in_row && c < A.N;
        const F8 f = widen8(h[u]), g = widen8(gm[u]);
        v4u y;
#pragma unroll
        for (int k = 0; k < 4; k++) y[k] = bf16x2(f.x[2 * k] * r * g.x[2 * k], f.x[2 * k + 1] * r * g.x[2 * k + 1]);
        if (A.y && in) store<kNTS>(reinterpret_cast<v4u*>(A.y + at + c), y);
        if (A.q) {   // a 1x32 block is a quad of lanes (G and N are multiples of a block's share)
            const F8 v = widen8(y);
            const uint32_t byte = mx_scale_byte(quad_max(absmax8_f32(v)));
            if (in) {
                store<kNTS>(reinterpret_cast<v2u*>(A.q + at + c), mx_encode8(v, ue8m0_operand(byte)));
                if ((t & 3) == 0) store_u8(A.e + (at + c) / 32, byte);
            }
        }
    }
}

// Workgroups walk the rows with a stride; gamma and the thread's columns of
// the dgamma sum stay in registers over all of them.
template <int G, int U>
__global__ __launch_bounds__(norm_threads(G)) void k_rmsnorm_grad(NormGradArgs A) {
    constexpr int TH = norm_threads(G), kRows = TH / G;
    __shared__ float lds[2][16];
    const int t = threadIdx.x % G;
    v4u gm[U];
    float dg[U][8];
#pragma unroll
    for (int u = 0; u < U; u++) {
        const int c = (u * G + t) * 8;
        gm[u] = c < A.N ? load<false>(reinterpret_cast<const v4u*>(A.gamma + c)) : v4u{};
#pragma unroll
        for (int k = 0; k < 8; k++) dg[u][k] = 0.0f;
    }
    const float inv_n = 1.0f / (float)A.N;
    int slot = 0;
    // whole workgroups step together: every thread reaches each row sum
    for (int64_t row0 = (int64_t)blockIdx.x * kRows; row0 < A.M; row0 += (int64_t)gridDim.x * kRows, slot ^= 1) {
        const int64_t row = row0 + threadIdx.x / G;
        const bool in_row = row < A.M;
        const int64_t at = row * A.N;
        v4u dy[U], h[U], dr[U];
#pragma unroll
        for (int u = 0; u < U; u++) {
            const int c = (u * G + t) * 8;
            const bool in = in_row && c < A.N;
            dy[u] = in ? load<kNTL>(reinterpret_cast<const v4u*>(A.dy + at + c)) : v4u{};
            h[u] = in ? load<kNTL>(reinterpret_cast<const v4u*>(A.h + at + c)) : v4u{};
            dr[u] = in && A.dres ? load<kNTL>(reinterpret_cast<const v4u*>(A.dres + at + c)) : v4u{};
        }
        const float r = in_row ? A.rstd[row] : 0.0f;
        float s = 0.0f;
#pragma unroll
        for (int u = 0; u < U; u++) {
            const F8 a = widen8(dy[u]), b = widen8(h[u]), g = widen8(gm[u]);
#pragma unroll
            for (int k = 0; k < 8; k++) {
                const float n = b.x[k] * r;
                s = __builtin_fmaf(a.x[k] * g.x[k], n, s);
                dg[u][k] = __builtin_fmaf(a.x[k], n, dg[u][k]);
            }
        }
        s = row_sum<G>(s, lds, slot) * inv_n;
#pragma unroll
        for (int u = 0; u < U; u++) {
            const int c = (u * G + t) * 8;
            const F8 a = widen8(dy[u]), b = widen8(h[u]), g = widen8(gm[u]), d = widen8(dr[u]);
            v4u o;
#pragma unroll
            for (int k = 0; k < 4; k++) {
                float p[2];
#pragma unroll
                for (int j = 0; j < 2; j++) {
                    const int i = 2 * k + j;
                    const float n = b.x[i] * r;
                    p[j] = __builtin_fmaf(r, __builtin_fmaf(-n, s, a.x[i] * g.x[i]), d.x[i]);
                }
                o[k] = bf16x2(p[0], p[1]);
            }
            if (in_row && c < A.N) store<kNTS>(reinterpret_cast<v4u*>(A.dx + at + c), o);
        }
    }
    if (!A.part) return;
    // the workgroup's partial sums: rows of one wave by lane exchanges, then wave
    // after wave through LDS (a fixed order: the result does not vary)
#pragma unroll
    for (int u = 0; u < U; u++)
#pragma unroll
        for (int k = 0; k < 8; k++)
#pragma unroll
            for (int x = G; x < 64; x *= 2) dg[u][k] += __shfl_xor(dg[u][k], x);
    float* part = A.part + (int64_t)blockIdx.x * A.N;
    if constexpr (G <= 64) {
        __shared__ __align__(16) float sum[G * U * 8];
        const int wave = threadIdx.x >> 6, lane = threadIdx.x & 63;
        for (int w = 0; w < TH / 64; w++) {
            if (wave == w && lane < G) {
#pragma unroll
                for (int u = 0; u < U; u++)
#pragma unroll
                    for (int k = 0; k < 8; k++) {
                        float* p = sum + (u * G + t) * 8 + k;
                        *p = w == 0 ? dg[u][k] : *p + dg[u][k];
                    }
            }
            __syncthreads();
        }
        for (int c = threadIdx.x; c < A.N; c += TH) part[c] = sum[c];
    } else {
#pragma unroll
        for (int u = 0; u < U; u++)
#pragma unroll
            for (int k = 0; k < 8; k++) {
                const int c = (u * G + t) * 8;
                if (c < A.N) part[c + k] = dg[u][k];
            }
    }
}

// dgamma[c] (+)= the sum of P partials in a fixed order: 32 threads of a column
// each take every 32nd partial, 8 loads at a time, then their sums are added in
// thread order.
constexpr int kDgCols = 32, kDgSlices = 32;
__global__ __launch_bounds__(kDgCols* kDgSlices) void k_rmsnorm_dgamma(const float* part, int32_t P, int32_t N, int accumulate,
                                                                      float* dgamma) {
    __shared__ float sum[kDgSlices][kDgCols];
    const int x = threadIdx.x % kDgCols, s = threadIdx.x / kDgCols;
    const int c = blockIdx.x * kDgCols + x;
    float a = 0.0f;
    if (c < N) {
#pragma unroll 8
        for (int p = s; p < P; p += kDgSlices) a += part[(int64_t)p * N + c];
    }
    sum[s][x] = a;
    __syncthreads();
    if (s == 0 && c < N) {
#pragma unroll
        for (int k = 1; k < kDgSlices; k++) a += sum[k][x];
        dgamma[c] = accumulate ? dgamma[c] + a : a;
    }
}

// Calls f(Threads per row, Vectors per thread) for rows of N elements: the
// smallest arrangement that holds the row.
template <int G, int U>
struct RowShape {
    static constexpr int g = G, u = U;
};
template <typename F>
auto by_row(int64_t N, F&& f) {
    const int64_t v = N / 8;   // 16-byte vectors of a row
    if (v <= 4) return f(RowShape<4, 1>{});
    if (v <= 8) return f(RowShape<8, 1>{});
    if (v <= 16) return f(RowShape<16, 1>{});
    if (v <= 32) return f(RowShape<32, 1>{});
    if (v <= 64) return f(RowShape<64, 1>{});
    if (v <= 128) return f(RowShape<64, 2>{});
    if (v <= 192) return f(RowShape<64, 3>{});
    if (v <= 256) return f(RowShape<64, 4>{});
    if (v <= 320) return f(RowShape<64, 5>{});
    if (v <= 384) return f(RowShape<64, 6>{});
    if (v <= 512) return f(RowShape<64, 8>{});
    if (v <= 768) return f(RowShape<256, 3>{});
    if (v <= 1024) return f(RowShape<256, 4>{});
    if (v <= 2048) return f(RowShape<1024, 2>{});
    return f(RowShape<1024, 4>{});
}

}  // namespace
