"""The Python functions over the entry points (csrc/calls.c) pass every argument on
as ctypes does, and refuse what is no number."""
import pytest

from test_expert_host import REFUSED as EXPERT
from test_mxfp4_host import REFUSED as MX
from tiled_dense_gemm_tma_b200 import binding, build as tg_build


@pytest.fixture(scope="module")
def calls():
    tg_build.build()
    return binding._calls()


@pytest.mark.parametrize("name,names,good,cases", EXPERT + MX, ids=[r[0] for r in EXPERT + MX])
def test_same_statuses(calls, name, names, good, cases):
    plain = getattr(binding.load_library(), name)
    for change, want in cases:
        a = dict(good, **change)
        args = [a[n] for n in names]
        assert getattr(calls, name)(*args) == plain(*args) == want, change


def test_every_call_of_the_binding_is_there(calls):
    import inspect
    import re
    text = inspect.getsource(binding)
    used = set(re.findall(r'_launch\("(tg_\w+)"', text))
    used |= {base + kind for base in ("tg_gemm_grouped_", "tg_gemm_grouped_wgrad_") for kind in ("f16", "bf16")}
    used = {u for u in used if not u.endswith("_")}
    assert used <= {n for n in dir(calls) if n.startswith("tg_")}
    assert "tg_expert_route" in used and "tg_gemm_mxfp4" in used and "tg_expert_sort" in used


def test_arguments_are_checked_for_number_and_kind(calls):
    with pytest.raises(TypeError):
        calls.tg_quant_i8(1, 2)
    with pytest.raises(TypeError):
        calls.tg_quant_mxfp4(0, 0, "x", 0, 0, None, 0, None, 0, None)
    with pytest.raises(TypeError):
        calls.tg_quant_mxfp4(0, 0, 1.5, 0, 0, None, 0, None, 0, None)
    with pytest.raises(OverflowError):
        calls.tg_quant_mxfp4(1 << 70, 0, None, 0, 0, None, 0, None, 0, None)
    with pytest.raises(TypeError):
        calls.tg_expert_route(0, 8, None, 8, 2, None, 0, 1, 1, 2, 1, "x", None, None, None)


def test_numbers_beyond_an_int_are_refused(calls):
    """Not cut to their lowest 32 bits, which could be a number that is allowed."""
    good = (0, 8, None, 8, 2, None, 0, 2, 1, 2, 1, 1.0, None, None, None)
    assert calls.tg_expert_route(*good) == 0
    for at in (1, 4, 6, 7, 8, 9, 10):
        for far in (1 << 32, -(1 << 32)):
            args = list(good)
            args[at] += far
            assert calls.tg_expert_route(*args) != 0, (at, far)
