"""The schedules that the 16-bit operators take for given sizes (host)."""

import ctypes

import bit_quantized_diffusion_amd as bq


def attention_plan(lens_q, lens_k, heads_q, heads_k, head_dim, causal):
    """(rows of a tile, parts, splits, workgroups of equal shares)"""
    plan = (ctypes.c_int32 * 4)()
    bq.check(bq.lib.svdq_debug_attention_plan(sum(lens_q), sum(lens_k), len(lens_q), heads_q, heads_k, head_dim, causal, plan))
    return tuple(plan)


def linear16_plan(m, n, k, aligned):
    """(rows of a tile, channels of a tile, waves, splits)"""
    plan = (ctypes.c_int32 * 4)()
    bq.check(bq.lib.svdq_debug_linear16_plan(m, n, k, aligned, plan))
    return tuple(plan)
