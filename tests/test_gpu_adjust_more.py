"""Adjusted logits that the other files do not look at: refused requests copied between
rows that lie differently, long histories."""
import pytest

from test_gpu_serve import BF, F32, request, sv          # noqa: F401
from test_gpu_adjust_removed import check_adjusted

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("in_elems,out_elems", [(0, 0), (1, 1), (0, 1), (3, 2), (5, 0)])
def test_refused_requests_of_unaligned_rows(sv, in_elems, out_elems, dtype):             # noqa: F811
    """A refused request's rows are copied as they are, not masked, wherever they lie."""
    for V in (4096, 5003):
        x, a = request(4, 3, V, 60, 43, biases=8, allowed=0.5, dtype=dtype)
        a["history_len"][:] = 60
        a["prompt_len"][:] = 7
        a["history"][1, 59] = V
        a["repetition"][3] = -1
        check_adjusted(sv, x, a, refused=(1, 3), in_elems=in_elems, out_elems=out_elems)


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("L", [8193, 40000, 131071])
def test_long_histories(sv, L, dtype):                # noqa: F811
    x, a = request(2, 3, 20003, L, L, biases=30, allowed=0.9, dtype=dtype)
    a["history_len"][0] = L
    a["prompt_len"][0] = L // 3
    check_adjusted(sv, x, a)
