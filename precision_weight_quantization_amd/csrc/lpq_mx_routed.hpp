// Products of microscaled matrices grouped by a plan: few rows (or short
// contractions) a group, from memory to registers.  The tiles of many rows are
// lpq_mx_matmul.hpp's.
//
// Part of lpq_kernels.hip, which includes each part once, in this order: one
// translation unit.
#pragma once

namespace {

// ROUTED_ROWS: y[r] = a[r] b[group of r]^T, for up to 16 * MT rows of one group and 16 * NT
// rows of its b.  ROUTED_K: y[g] = a[:, rows of g] b[:, rows of g]^T, 16 * MT rows of a, 16 * NT
// of b.  W waves share out k in steps of 128 and add their results through LDS; a
// workgroup holds 8 / W such tiles side by side, because a wave of few steps spends its time
// on finding its group and on one round trip to memory.  Memory is the floor, the weights of the groups that
// have rows: 24 tokens of 8 experts, N = 2048, k = 768, MXFP4 weights 15 us, 5.5 TB/s where the routing reaches 100 of 128
// groups and four sets of weights take turns; N = 1536, k = 2048 in MXFP8 71 us, 4.4 TB/s from memory.
template <bool FP4B, bool FP4A, int NT, int MT, int U, int W, TileMode MODE>
__global__ __launch_bounds__(64 * kRowsWaves) void k_mx_matmul_routed_rows(MatmulArgs A, int tiles_n, int tiles_m, Routing routing,
                                                                           int first) {
    constexpr int C = kRowsWaves / W;   // column tiles of the workgroup
    __shared__ v4f parts[C][W][NT * MT][64];
    const int lane = threadIdx.x & 63, g = lane >> 4, r = lane & 15;
    const int wave = (threadIdx.x >> 6) % W, column = (threadIdx.x >> 6) / W;
    auto& part = parts[column];
    int tile = first + (int)blockIdx.x, group, k0 = 0, K = A.K;
    int64_t m_first, m_last;
    if constexpr (MODE == ROUTED_ROWS) {
        const RouteMap map(routing, RowTiles<16 * MT>{});
        const int v = tile / tiles_n;
        if (v >= map.total) return;   // the whole workgroup: the grid is for the most tiles there may be
        RouteRun r;
        int within;
        group = map.find(routing, v, r, within);
        m_first = r.first + within * 16 * MT;
        m_last = min(r.first + (within + 1) * 16 * MT, r.last);
    } else {
        group = tile / (tiles_n * tiles_m);
        tile -= group * tiles_n * tiles_m;
        const RouteRun run = wave_run(routing, group);
        k0 = run.first / 32 * 32;   // whole blocks: a plan with align 32 has no others
        K = run.last / 32 * 32 - k0;
        m_first = (int64_t)(tile / tiles_n) * 16 * MT;
        m_last = A.M;
    }
    const int64_t n_first = ((int64_t)(tile % tiles_n) * C + column) * 16 * NT, b_first = MODE == ROUTED_ROWS ? (int64_t)group * A.N : 0;
    const uint8_t *a[MT], *ae[MT], *b[NT], *be[NT];
    bool in_m[MT], in_n[NT];
    v4f c[NT][MT];
#pragma unroll
    for (int j = 0; j < NT; j++) {
        const int64_t n = n_first + j * 16 + r;
        in_n[j] = n < A.N;
        const int64_t row = b_first + (in_n[j] ? n : 0);
        b[j] = A.b + row * row_bytes<FP4B>(A.K) + row_bytes<FP4B>(k0);
        be[j] = A.be + row * (A.K / 32) + k0 / 32;
    }
#pragma unroll
    for (int i = 0; i < MT; i++) {
        const int64_t m = m_first + i * 16 + r;
        in_m[i] = m < m_last;
        const int64_t row = in_m[i] ? m : m_first;
        a[i] = A.a + row * row_bytes<FP4A>(A.K) + row_bytes<FP4A>(k0);
        ae[i] = A.ae + row * (A.K / 32) + k0 / 32;
#pragma unroll
        for (int j = 0; j < NT; j++) c[j][i] = v4f{0.0f, 0.0f, 0.0f, 0.0f};
    }
    for (int k = wave * 128; k < K; k += W * 128 * U) {
        Frag<FP4B> fb[U][NT];
        Frag<FP4A> fa[U][MT];
#pragma unroll
        for (int u = 0; u < U; u++) {
            const int at = k + u * W * 128;
#pragma unroll
            for (int j = 0; j < NT; j++) fb[u][j] = load_frag<FP4B>(b[j], be[j], in_n[j], at, K, g);
#pragma unroll
            for (int i = 0; i < MT; i++) fa[u][i] = load_frag<FP4A>(a[i], ae[i], in_m[i], at, K, g);
        }
#pragma unroll
        for (int u = 0; u < U; u++)
#pragma unroll
            for (int j = 0; j < NT; j++)
#pragma unroll
                for (int i = 0; i < MT; i++) c[j][i] = mfma<FP4B, FP4A>(fb[u][j], fa[u][i], c[j][i]);
    }
#pragma unroll
    for (int j = 0; j < NT; j++)
#pragma unroll
        for (int i = 0; i < MT; i++) part[wave][j * MT + i][lane] = c[j][i];
    __syncthreads();
    for (int x = wave; x < NT * MT; x += W) {
        v4f s = part[0][x][lane];
#pragma unroll
        for (int w = 1; w < W; w++) s += part[w][x][lane];
        const int64_t m = m_first + x % MT * 16 + r, n = n_first + x / MT * 16 + g * 4;
        if (m < m_last && n < A.N) store_y4(A, MODE == ROUTED_ROWS ? m : (int64_t)group * A.M + m, (int)n, s);
    }
}

}  // namespace
