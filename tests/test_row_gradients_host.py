"""What the zeros of unnamed rows refuse, without a GPU."""
import pytest

from moe_ragged_grouped_gb300 import build as gg_build
from moe_ragged_grouped_gb300 import cake_gg as gg

AT = 1 << 20
INVALID, ALIGN, KIND, OVER = gg.CAKE_GG_ERR_INVALID_ARG, gg.CAKE_GG_ERR_ALIGNMENT, gg.CAKE_GG_ERR_UNSUPPORTED, gg.CAKE_GG_ERR_OVERFLOW


@pytest.mark.parametrize("change,code", [
    (dict(T=-1), INVALID), (dict(M=-1), INVALID), (dict(M=2 ** 31), INVALID), (dict(top_k=0), INVALID), (dict(top_k=33), INVALID),
    (dict(K=12), ALIGN), (dict(K=2 ** 20 + 8), OVER), (dict(rows_dtype=2), KIND), (dict(position=None), INVALID), (dict(rows=None), INVALID),
    (dict(named=None), INVALID), (dict(rows=AT + 8), ALIGN), (dict(position=AT + 2), ALIGN), (dict(M=0), gg.CAKE_GG_OK),
])
def test_refuses(change, code):
    gg_build.build()
    a = dict(T=4, M=8, top_k=2, K=64, position=AT, rows=AT, rows_dtype="bf16", named=AT, stream=0)
    a.update(change)
    assert gg.cake_gg_zero_unnamed_rows(**a) == code
