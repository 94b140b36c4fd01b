"""Refusals of linear_form, before any device call.  CPU-only."""

import ctypes

import pytest
import torch

from block_scaled_fp8_route_gb300 import _lib, build, ops


def test_statuses():
    lib = _lib.load(build.build())
    form = (ctypes.c_int64 * 4)()
    for bad in ((0, 8, 8, 1, 0, form), (-1, 8, 8, 1, 0, form), (4, 0, 8, 1, 0, form), (4, 8, 0, 1, 0, form),
                (4, 8, 8, 2, 0, form), (4, 8, 8, -1, 0, form), (4, 8, 8, 1, 0, None)):
        assert lib.bsf_linear_form(*bad) == 1, bad
    for bad in ((2 ** 31, 8, 8, 1, 0, form), (4, 2 ** 25, 8, 1, 0, form), (4, 8, 2 ** 25, 1, 0, form)):
        assert lib.bsf_linear_form(*bad) == 3, bad


def test_types_of_torch():
    _lib.load(build.build())
    with pytest.raises(_lib.BsfError):
        ops.linear_form(4, 8, 8, torch.int32)
