// Operands and epilogue of the dense products, as their kernels take them.
#pragma once
#include <cuda.h>

#include "common.cuh"
#include "launch.h"

namespace la {

struct Maps {
    CUtensorMap a[2], b[2];
};

struct Epilogue {
    __nv_bfloat16 *out[2];
    const __nv_bfloat16 *bias, *residual;
    __nv_bfloat16 *saved;  // LINEAR: z [M][lds]; GATED: upper 16 bits of gate | up [M][lds], up from column half on
    uint8_t *lower;        // GATED: the next eight bits, laid out the same
    int64_t ldo[2], ldr, lds;
    int half, act;
    float *partial;  // DW split: [out][part][M][ldp] fp32
    int64_t ldp;
};

// Tensor maps of a call's operands. An operand that runs along the summed index is read in boxes of 64 of its
// columns x 64 summed rows (MN-major), any other in boxes of 64 summed columns x box_a (box_b) rows.
inline bool make_maps(Maps *maps, const DenseArgs &a, bool a_mn, bool b_mn, uint32_t box_a, uint32_t box_b) {
    const int na = a.kind == DENSE_DX || a.kind == DENSE_DW ? a.count : 1;
    const int nb = a.kind == DENSE_GATED ? 2 : a.kind == DENSE_DX ? a.count : 1;
    for (int i = 0; i < na; ++i)
        if (!(a_mn ? make_map_bf16_2d(&maps->a[i], a.a[i], a.K, a.M, a.lda[i], 64, 64, true)
                   : make_map_bf16_2d(&maps->a[i], a.a[i], a.M, a.K, a.lda[i], 64, box_a, true)))
            return false;
    for (int i = 0; i < nb; ++i)
        if (!(b_mn ? make_map_bf16_2d(&maps->b[i], a.b[i], a.K, a.N, a.ldb[i], 64, 64, true)
                   : make_map_bf16_2d(&maps->b[i], a.b[i], a.N, a.K, a.ldb[i], 64, box_b, true)))
            return false;
    if (na == 1) maps->a[1] = maps->a[0];
    if (nb == 1) maps->b[1] = maps->b[0];
    return true;
}

inline Epilogue make_epilogue(const DenseArgs &a) {
    Epilogue ep{};
    for (int i = 0; i < 2; ++i) {
        ep.out[i] = (__nv_bfloat16 *)a.out[i];
        ep.ldo[i] = a.ldo[i];
    }
    ep.bias = (const __nv_bfloat16 *)a.bias;
    ep.residual = (const __nv_bfloat16 *)a.residual;
    ep.saved = (__nv_bfloat16 *)a.saved;
    ep.lower = (uint8_t *)a.lower;
    ep.ldr = a.ldr;
    ep.lds = a.lds;
    ep.half = a.half;
    ep.act = a.act;
    ep.partial = a.partial;
    ep.ldp = ((int64_t)a.N + 7) / 8 * 8;
    return ep;
}

}  // namespace la
