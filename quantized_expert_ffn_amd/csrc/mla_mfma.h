// Matrix-core operations of the latent-attention kernels on gfx950, in
// bfloat16 and binary16 with binary32 accumulation, and what feeds them.
//
// v_mfma_f32_32x32x16: C[32x32] += A[32x16] B[16x32].  Lane layout:
//   A: lane l holds A[i][k], i = l % 32, k = 8 (l / 32) + j, in element j;
//   B: lane l holds B[k][n], n = l % 32, k likewise;
//   C: register r of lane l holds C[i][n], n = l % 32,
//      i = 8 (r / 4) + 4 (l / 32) + r % 4.
// The kernels form transposed scores S^T = K Q^T, so that a lane holds sixteen
// keys of one query: its softmax needs one exchange between the lane halves.
// Registers 8 s .. 8 s + 7 are then, as they stand, the B operand of O^T +=
// V^T P^T if element j of the A operand's lane half h is the value of key
// 16 s + 8 (j / 4) + 4 h + j % 4: the transposing LDS reads take a row address
// a lane, so that order costs nothing and P never leaves its registers.
#pragma once

#include "mla_common.h"

namespace coli {

typedef float f32x16 __attribute__((ext_vector_type(16)));
typedef short s16x4 __attribute__((ext_vector_type(4)));

template <class T>
__device__ __forceinline__ f32x16 mfma32(x8<T> a, x8<T> b, f32x16 c);
template <>
__device__ __forceinline__ f32x16 mfma32<__bf16>(x8<__bf16> a, x8<__bf16> b, f32x16 c) {
    return __builtin_amdgcn_mfma_f32_32x32x16_bf16(a, b, c, 0, 0, 0);
}
template <>
__device__ __forceinline__ f32x16 mfma32<_Float16>(x8<_Float16> a, x8<_Float16> b, f32x16 c) {
    return __builtin_amdgcn_mfma_f32_32x32x16_f16(a, b, c, 0, 0, 0);
}

// LDS is addressed by byte offset from the start of the workgroup's dynamic
// allocation, which begins at offset 0: the kernels declare no static LDS and
// call nothing that has some (a barrier that carries a value does).
// `imm` is a constant the instruction's offset field takes.
template <class V>
__device__ __forceinline__ V lds_read(uint32_t off, int imm = 0) {
    return *(const __attribute__((address_space(3))) V *)((const __attribute__((address_space(3))) char *)off + imm);
}
template <class V>
__device__ __forceinline__ void lds_write(uint32_t off, V v, int imm = 0) {
    *(__attribute__((address_space(3))) V *)((__attribute__((address_space(3))) char *)off + imm) = v;
}

// Transposing reads.  Sixteen lanes read a block of rows of 16 columns and
// each receives one column: 16-bit elements, four rows, lane x reading columns
// 4 (x % 4) .. + 3 of row x / 4; bytes, eight rows, lane x reading columns
// 8 (x % 2) .. + 7 of row x / 2.
__device__ __forceinline__ u32x2 lds_read_tr16(uint32_t off, int imm) {
    typedef __attribute__((address_space(3))) s16x4 lds_v;
    return __builtin_bit_cast(u32x2, __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_v *)((__attribute__((address_space(3))) char *)off + imm)));
}
__device__ __forceinline__ u32x2 lds_read_tr8(uint32_t off, int imm) {
    typedef int i32x2 __attribute__((ext_vector_type(2)));
    typedef __attribute__((address_space(3))) i32x2 lds_v;
    return __builtin_bit_cast(u32x2, __builtin_amdgcn_ds_read_tr8_b64_v2i32((lds_v *)((__attribute__((address_space(3))) char *)off + imm)));
}

// Eight E4M3 codes as eight values of T: exact in both types (four
// significant bits, exponents -9 .. 8).
template <class T>
__device__ __forceinline__ x8<T> widen8(u32x2 c);
template <>
__device__ __forceinline__ x8<__bf16> widen8<__bf16>(u32x2 c) {
    x8<__bf16> o;
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        const x2<__bf16> a = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(c[i], 1.0f, false);
        const x2<__bf16> b = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(c[i], 1.0f, true);
        o[4 * i] = a[0];
        o[4 * i + 1] = a[1];
        o[4 * i + 2] = b[0];
        o[4 * i + 3] = b[1];
    }
    return o;
}
template <>
__device__ __forceinline__ x8<_Float16> widen8<_Float16>(u32x2 c) {
    x8<_Float16> o;
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        const x2<_Float16> a = __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(c[i], 1.0f, false);
        const x2<_Float16> b = __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(c[i], 1.0f, true);
        o[4 * i] = a[0];
        o[4 * i + 1] = a[1];
        o[4 * i + 2] = b[0];
        o[4 * i + 3] = b[1];
    }
    return o;
}

// The larger of a lane's value and the other lane half's.
__device__ __forceinline__ float half_max(float v) {
    const auto r = __builtin_amdgcn_permlane32_swap(__float_as_uint(v), __float_as_uint(v), false, false);
    return fmaxf(__uint_as_float(r[0]), __uint_as_float(r[1]));
}
__device__ __forceinline__ float half_sum(float v) {
    const auto r = __builtin_amdgcn_permlane32_swap(__float_as_uint(v), __float_as_uint(v), false, false);
    return __uint_as_float(r[0]) + __uint_as_float(r[1]);
}

// Softmax weights are rounded to T in units of 2^-LIFT of the running maximum's.
// binary16 has no normal number below 2^-14 and none below 2^-24: relative to
// the maximum itself, 10^5 keys of 2^-26 each would vanish, 2^-9 of the sum.
// Lifted by 2^7 they do from 2^-32 on, and the maximum's lag still fits.
template <class T>
inline constexpr float WEIGHT_LIFT = 0.0f;
template <>
inline constexpr float WEIGHT_LIFT<_Float16> = 7.0f;

// Inclusive sums over the wavefront (shifts within 16 lanes, then broadcasts
// of the rows before).
template <int CTRL, int ROWS>
__device__ __forceinline__ int dpp_add(int v) {
    return v + __builtin_amdgcn_update_dpp(0, v, CTRL, ROWS, 0xf, false);
}
__device__ __forceinline__ int wave_scan(int v) {
    v = dpp_add<0x111, 0xf>(v);
    v = dpp_add<0x112, 0xf>(v);
    v = dpp_add<0x114, 0xf>(v);
    v = dpp_add<0x118, 0xf>(v);
    v = dpp_add<0x142, 0xa>(v);
    return dpp_add<0x143, 0xc>(v);
}

// t / d for 0 <= t < 2^31 with inv = (2^32 - 1) / d: the product falls short
// of the quotient by one at most.
__device__ __forceinline__ int div_by(int t, int d, uint32_t inv) {
    const int q = (int)__umulhi((uint32_t)t, inv);
    return t - q * d >= d ? q + 1 : q;
}

// 16 bytes of each lane straight into LDS: from src + OFF, lane l's to lds +
// lds_off + 16 l (lds uniform over the wavefront).  Done when the wavefront's
// vmcnt says so.  Written in assembly because the compiler otherwise waits for
// every such load before the next LDS read of any buffer; no register is an
// output.  The instruction's offset counts on both sides, hence the
// subtraction; the wait state is the one between a write of m0 and a load that
// reads it.
template <int OFF = 0>
__device__ __forceinline__ void load_to_lds(const void *src, uint32_t lds, int lds_off = 0) {
    asm volatile("s_add_u32 m0, %1, %2\n\ts_nop 0\n\tglobal_load_lds_dwordx4 %0, off offset:%3" ::"v"(src),
                 "s"(__builtin_amdgcn_readfirstlane((int)lds)), "i"(lds_off - OFF), "n"(OFF)
                 : "memory", "scc", "m0");
}

// The same from a base all lanes share and an offset of each.  Five wait
// states pass before the load, what it needs if a vector instruction has just
// written the base.
template <int OFF>
__device__ __forceinline__ void load_to_lds_from(const void *base, uint32_t at, uint32_t lds, int lds_off) {
    asm volatile("s_add_u32 m0, %2, %3\n\ts_nop 3\n\tglobal_load_lds_dwordx4 %0, %1 offset:%4" ::"v"(at), "s"(base),
                 "s"(__builtin_amdgcn_readfirstlane((int)lds)), "i"(lds_off - OFF), "n"(OFF)
                 : "memory", "scc", "m0");
}

// A 32-bit word of each lane straight into LDS, lane l's to lds + 4 l.
__device__ __forceinline__ void load_word_to_lds(const void *src, uint32_t lds) {
    asm volatile("s_mov_b32 m0, %1\n\ts_nop 0\n\tglobal_load_lds_dword %0, off" ::"v"(src),
                 "s"(__builtin_amdgcn_readfirstlane((int)lds))
                 : "memory", "m0");
}

// A value that is the same in every lane, as a scalar.
__device__ __forceinline__ int uniform(int v) { return __builtin_amdgcn_readfirstlane(v); }

// Waits until at most N of the wavefront's vector-memory operations are out.
template <int N>
__device__ __forceinline__ void wait_vm() {
    static_assert(N < 64, "vmcnt has six bits");
    asm volatile("s_waitcnt vmcnt(%0)" ::"n"(N) : "memory");
}

// Makes the compiler wait for a value it loaded here, not at its first use.
template <class V>
__device__ __forceinline__ void arrived(V &v) {
    asm volatile("" : "+v"(v));
}

// The same for a matrix operand that is to stay in an accumulation register:
// the matrix instructions read it there.
template <class V>
__device__ __forceinline__ void arrived_acc(V &v) {
    asm volatile("" : "+a"(v));
}

// A workgroup barrier that waits for this wavefront's LDS accesses, but not
// for its loads from memory.
__device__ __forceinline__ void barrier_lds() {
    asm volatile("s_waitcnt lgkmcnt(0)\n\ts_barrier" ::: "memory");
}

}  // namespace coli
