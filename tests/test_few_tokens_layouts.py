"""Unquantised weights of few_token_moe: tensors of dtype bfloat16 are rows whatever the flags say, bytes are what the flags
say, and the two do not mix under ``B_TILED``.  CPU-only."""

import pytest

from block_scaled_fp8_route_gb300 import ops
from tests.test_few_tokens_refusals import BF16, U8, Library, Reached, Tensor, library, moe, moe_operands  # noqa: F401

ROWS = dict(w13=Tensor(8, 256, 256, dtype=BF16), w2=Tensor(8, 256, 128, dtype=BF16),
            shared_w13=Tensor(512, 256, dtype=BF16), shared_w2=Tensor(256, 256, dtype=BF16))


@pytest.fixture
def flags(library, monkeypatch):  # noqa: F811
    seen = []

    def call(*a):
        seen.append(a[-2])
        raise Reached
    monkeypatch.setattr(Library, "bsf_few_token_moe", staticmethod(call))
    return seen


def call(t, **kw):
    shared = None if t["shared_w13"] is None else tuple(t["shared_" + k] for k in ("w13", "sfb13", "w2", "sfb2"))
    with pytest.raises(Reached):
        ops.few_token_moe(t["x"], t["topk_ids"], t["topk_weights"], t["w13"], t["sfb13"], t["w2"], t["sfb2"], shared=shared,
                          z=t["z"], workspace=t["workspace"], **kw)


@pytest.mark.parametrize("shared", [True, False])
def test_rows_are_read_as_rows(flags, shared):
    t = moe_operands(BF16, **ROWS)
    if not shared:
        t["shared_w13"] = None
    call(t)
    call(t, flags=0)
    call(t, flags=ops.B_TILED | 0x100)
    assert flags == [0, 0, 0x100]


def test_bytes_are_read_as_the_flags_say(flags):
    for kind in (BF16, U8):
        call(moe_operands(kind))
        call(moe_operands(kind), flags=0)
    assert flags == [ops.B_TILED, 0] * 2
    call(moe_operands(BF16, w2=ROWS["w2"]), flags=0)             # (all rows)
    assert flags[-1] == 0


@pytest.mark.parametrize("name", list(ROWS))
def test_rows_do_not_mix_with_tiled_bytes(flags, name):
    with pytest.raises(ValueError, match="tile_weights"):
        moe(moe_operands(BF16, **{name: ROWS[name]}))
    with pytest.raises(ValueError, match="tile_weights"):
        moe(moe_operands(BF16, **{k: v for k, v in ROWS.items() if k != name}))
