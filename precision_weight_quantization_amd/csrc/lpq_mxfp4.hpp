// MXFP4: quantize (default and floor exponent rules), dequantize and QDQ.
//
// Streaming work bound by memory: 2 bytes in and 17/32 out an element, the other way
// round, or 2 and 2.  Measured at 9728 x 2560, buffers larger than the memory-side cache:
// quantize 11.9 us and dequantize 12.3 (63 MB, 5.1 to 5.3 TB/s, the rate of a large copy),
// fake-quantize 17.9 (100 MB, 5.6 TB/s); 128 tensors of 768 x 2048 in a grouped call 79, 90
// and 126 us (5.7 to 6.5 TB/s).
//
// Part of lpq_kernels.hip, which includes each part once, in this order: one
// translation unit.
#pragma once

namespace {

// ---------------------------------------------------------------------------
// MXFP4
// ---------------------------------------------------------------------------

// Scale byte of a block amax given as binary32 bits (a BF16 value): the
// smallest e with amax <= 6 * 2^e (6 = 1.5 * 2^2), biased by 127.  Adding 63 to
// the 7-bit mantissa field carries into the exponent exactly when it is above
// 64, the mantissa of 1.5.
__device__ __forceinline__ uint32_t mx4_scale_byte(uint32_t amax_bits) {
    const int e = (int)((amax_bits + (63u << 16)) >> 23) - 2;
    return (uint32_t)(e > 0 ? e : 0);
}

// The floor rule: byte = max(0, floor(log2 amax) - 2 + 127).  Elements up to
// 8 * 2^e are left for the saturating cast.
__device__ __forceinline__ uint32_t mx4_floor_scale_byte(uint32_t amax_bits) {
    const int e = (int)(amax_bits >> 23) - 2;
    return (uint32_t)(e > 0 ? e : 0);
}

template <bool FLOOR>
__device__ __forceinline__ uint32_t mx4_byte(uint32_t amax_bits) {
    return FLOOR ? mx4_floor_scale_byte(amax_bits) : mx4_scale_byte(amax_bits);
}

// 8 BF16 values -> 8 E2M1 codes of RN(x / 2^(byte - 127)), saturating, X
// carrying the byte (one word, element 0 in the low nibble).  The conversion
// takes a packed pair of BF16 and keeps the sign of zero.
__device__ __forceinline__ uint32_t mx4_encode8(const v4u& v, float X) {
    // words of their own first: a bit cast of a vector's element takes its element 0
    const uint32_t a = v.x, b = v.y, c = v.z, d = v.w;
    uint32_t p = a;   // every byte is written: it starts from any value
    p = __builtin_amdgcn_cvt_scalef32_pk_fp4_bf16(p, __builtin_bit_cast(bf16x2_t, a), X, 0);
    p = __builtin_amdgcn_cvt_scalef32_pk_fp4_bf16(p, __builtin_bit_cast(bf16x2_t, b), X, 1);
    p = __builtin_amdgcn_cvt_scalef32_pk_fp4_bf16(p, __builtin_bit_cast(bf16x2_t, c), X, 2);
    p = __builtin_amdgcn_cvt_scalef32_pk_fp4_bf16(p, __builtin_bit_cast(bf16x2_t, d), X, 3);
    return p;
}

// 8 E2M1 codes times 2^(byte - 127) -> 8 BF16 values.
__device__ __forceinline__ v4u mx4_decode8(uint32_t p, float X) {
    v4u o;
    o.x = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(p, X, 0));
    o.y = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(p, X, 1));
    o.z = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(p, X, 2));
    o.w = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(p, X, 3));
    return o;
}

// The flat layout of the MXFP8 kernels: a quad of lanes is one 32-element
// block, 16 bytes of BF16 in and 4 bytes of codes out per lane.
template <int U, int TH, bool GROUPED, bool FLOOR = false, bool AHEAD = LPQ_MX4Q_AHEAD != 0>
__global__ __launch_bounds__(TH) void k_mxfp4_quant(const lpq_tensor* table, lpq_tensor one, ChunkMap map) {
    const Work W = locate<GROUPED>(table, one, map);
    const lpq_tensor& d = W.d;
    const int64_t total = d.rows * d.cols;
    const int64_t base = W.unit * chunk_elems<U, TH>();
    const v4u* src = reinterpret_cast<const v4u*>(d.src);
    uint32_t* dst = reinterpret_cast<uint32_t*>(d.dst);
    uint8_t* esc = reinterpret_cast<uint8_t*>(d.scale);
    const int tid = threadIdx.x;
    by_fullness<chunk_elems<U, TH>()>(base, total, [&](auto full) {
        constexpr bool FULL = decltype(full)::value;
        v4u v[U];
        auto fetch = [&](int u) { v[u] = load_vec<TH, FULL>(src, base, total, u); };
        fetch_start<U, AHEAD>(fetch);
#pragma unroll
        for (int u = 0; u < U; u++) {
            fetch_step<U, AHEAD>(u, fetch, v[u].x);
            const int64_t e0 = base + (int64_t)(u * TH + tid) * 8;
            const uint32_t byte = mx4_byte<FLOOR>(quad_max(absmax8_bits(v[u])));
            const uint32_t codes = mx4_encode8(v[u], ue8m0_operand(byte));
            if (FULL || e0 < total) {
                store<kNTS>(dst + (e0 >> 3), codes);
                if ((tid & 3) == 0) store_u8(esc + (e0 >> 5), byte);
            }
        }
    });
}

template <int U, int TH, bool GROUPED, bool AHEAD = LPQ_MX4D_AHEAD != 0>
__global__ __launch_bounds__(TH) void k_mxfp4_dequant(const lpq_tensor* table, lpq_tensor one, ChunkMap map) {
    const Work W = locate<GROUPED>(table, one, map);
    const lpq_tensor& d = W.d;
    const int64_t total = d.rows * d.cols;
    const int64_t base = W.unit * chunk_elems<U, TH>();
    const uint32_t* src = reinterpret_cast<const uint32_t*>(d.src);
    v4u* dst = reinterpret_cast<v4u*>(d.dst);
    const uint8_t* esc = reinterpret_cast<const uint8_t*>(d.scale);
    const int tid = threadIdx.x;
    by_fullness<chunk_elems<U, TH>()>(base, total, [&](auto full) {
        constexpr bool FULL = decltype(full)::value;
        uint32_t c[U], b[U];
        auto fetch = [&](int u) {
            const int64_t e0 = base + (int64_t)(u * TH + tid) * 8;
            c[u] = load_vec<TH, FULL>(src, base, total, u);
            b[u] = (FULL || e0 < total) ? load_u8(esc + (e0 >> 5)) : 127u;
        };
        fetch_start<U, AHEAD>(fetch);
#pragma unroll
        for (int u = 0; u < U; u++) {
            fetch_step<U, AHEAD>(u, fetch, c[u], b[u]);
            const int64_t e0 = base + (int64_t)(u * TH + tid) * 8;
            const v4u o = mx4_decode8(c[u], ue8m0_operand(b[u]));
            if (FULL || e0 < total) store<kNTS>(dst + (e0 >> 3), o);
        }
    });
}

template <int U, int TH, bool GROUPED, bool FLOOR = false, bool AHEAD = LPQ_MX4QDQ_AHEAD != 0>
__global__ __launch_bounds__(TH) void k_mxfp4_qdq(const lpq_tensor* table, lpq_tensor one, ChunkMap map) {
    const Work W = locate<GROUPED>(table, one, map);
    const lpq_tensor& d = W.d;
    const int64_t total = d.rows * d.cols;
    const int64_t base = W.unit * chunk_elems<U, TH>();
    const v4u* src = reinterpret_cast<const v4u*>(d.src);
    v4u* dst = reinterpret_cast<v4u*>(d.dst);
    const int tid = threadIdx.x;
    by_fullness<chunk_elems<U, TH>()>(base, total, [&](auto full) {
        constexpr bool FULL = decltype(full)::value;
        v4u v[U];
        auto fetch = [&](int u) { v[u] = load_vec<TH, FULL>(src, base, total, u); };
        fetch_start<U, AHEAD>(fetch);
#pragma unroll
        for (int u = 0; u < U; u++) {
            fetch_step<U, AHEAD>(u, fetch, v[u].x);
            const int64_t e0 = base + (int64_t)(u * TH + tid) * 8;
            const float X = ue8m0_operand(mx4_byte<FLOOR>(quad_max(absmax8_bits(v[u]))));
            const v4u o = mx4_decode8(mx4_encode8(v[u], X), X);
            if (FULL || e0 < total) store<kNTS>(dst + (e0 >> 3), o);
        }
    });
}

}  // namespace
