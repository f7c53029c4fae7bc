"""The schedules of the 16-bit operators, on the host: what the test hooks
refuse, and that the GPU tests' sizes reach every kernel."""

import ctypes

import pytest

import bit_quantized_diffusion_amd as bq
from tests import test_gpu_attention_rows as rows
from tests import test_gpu_attention_wide as wide
from tests import test_gpu_linear16_tiles as tiles
from tests._plans import attention_plan, linear16_plan

BAD, SHAPE = bq.SVDQ_ERR_INVALID_ARG, bq.SVDQ_ERR_SHAPE


def test_hooks_refuse():
    plan = (ctypes.c_int32 * 4)()
    a, l = bq.lib.svdq_debug_attention_plan, bq.lib.svdq_debug_linear16_plan
    assert a(1, 1, 1, 1, 1, 64, 0, None) == BAD and l(1, 1, 1, 0, None) == BAD
    assert a(1, 1, 0, 1, 1, 64, 0, plan) == SHAPE and a(1, 1, 1, 3, 2, 64, 0, plan) == SHAPE and a(1, 1, 1, 1, 1, 60, 0, plan) == SHAPE
    assert l(0, 1, 8, 0, plan) == SHAPE and l(1, 1, 9, 1, plan) == SHAPE


def test_attention_sizes_reach_every_schedule():
    assert len(rows.SCHEDULES) == len(rows.PLANS)
    for case, want in zip(rows.SCHEDULES, rows.PLANS):
        height, parts, splits, shares = attention_plan(*case)
        assert (height, parts, splits > 1, shares > 0) == want, case
    for case in wide.CASES:
        assert attention_plan(*case, False) == (256, 1, 1, 0), case


def test_linear16_sizes_reach_every_tile_shape():
    for case, want in tiles.TILES.items():
        assert linear16_plan(*case) == want, case
    shapes = {(c[3], *p[:3], p[3] > 1) for c, p in tiles.TILES.items()}
    assert len(shapes) >= 11


@pytest.mark.parametrize("m,n,waves", [(1, 64, 4), (8, 20000, 4), (9, 8192, 4), (9, 8193, 2), (32, 20000, 2)])
def test_few_rows(m, n, waves):
    assert linear16_plan(m, n, 512, True) == (32, 32, waves, 1)
