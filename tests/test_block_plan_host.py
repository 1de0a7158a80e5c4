"""How kv8_attention divides its work (csrc/kv8_plan.hpp, host code in the library): each division that
the GPU tests name is the one that its sizes get, so that none loses its tests when a threshold
moves."""

import ctypes

import pytest

from bit_codebook_quantized_amd import w4a8
from test_gpu_block_attention_divisions import DIVISIONS

I64, INT, BOOL = ctypes.c_int64, ctypes.c_int, ctypes.c_bool


class Plan(ctypes.Structure):
    """Mirror of struct AttentionPlan."""
    _fields_ = [("rows", INT), ("prompt", BOOL), ("tiles", I64), ("halves", BOOL), ("wide", BOOL), ("parts", BOOL),
                ("chunks", INT), ("chunk_steps", INT), ("blocks", I64), ("join_blocks", I64), ("part_rows", I64)]


def plan(lens, news, q_heads, kv_heads, head_dim):
    fn = getattr(ctypes.CDLL(w4a8.LIB_PATH), "_ZN4w4a814attention_planEllliii")     # w4a8::attention_plan
    fn.argtypes, fn.restype = [I64] * 3 + [INT] * 3, Plan
    return fn(len(lens), max(news), max(lens), q_heads, kv_heads, head_dim)


# name: rows of a block, wide, halves, parts
WANT = {
    "one launch": (16, True, False, False),
    "16 rows, a block a pair": (16, False, False, False),
    "16 rows, dealt": (16, False, False, True),
    "64 rows": (64, False, True, False),
    "64 rows, many pairs": (64, False, False, False),
    "64 rows in chunks": (64, False, False, True),
    "128 rows": (128, False, False, False),
    "128 rows in chunks": (128, False, False, True),
}


@pytest.mark.parametrize("head_dim", [64, 128])
@pytest.mark.parametrize("name", DIVISIONS)
def test_division_is_the_one_that_its_name_says(name, head_dim):
    p = plan(*DIVISIONS[name], head_dim)
    assert (p.rows, p.wide, p.halves, p.parts) == WANT[name]
    assert p.prompt == (p.rows > 16) and (p.chunks > 1) == (p.prompt and p.parts)


def test_every_division_has_a_name():
    """What launch_attention distinguishes: 16 rows wide, dealt or not; 64 in halves, chunks or neither; 128 in chunks or not."""
    assert set(WANT) == set(DIVISIONS) and len(set(WANT.values())) == 8
