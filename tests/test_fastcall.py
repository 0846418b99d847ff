"""CPU: the binding's call module converts arguments as the C ABI takes them and refuses others."""
import ctypes

import pytest

import long_context_layer_b200 as L
from long_context_layer_b200 import _native as N

# a function of sixteen words at most that only looks at its first arguments: sel_capacity(params, page_size)
CAP = ctypes.cast(N.lib.delta_sel_capacity, ctypes.c_void_p).value


def test_structure_and_integer_arguments():
    f = N._bind("cap", CAP, (L.DeltaSelectParams, "i"))
    sp = L.DeltaSelectParams(64, 16, 256, 0)
    assert f(sp, 16) == L.sel_capacity(sp) == 82
    assert f(sp, -1) == -1                       # negative integers arrive as they are
    sp.budget_pages = 5
    assert f(sp, 16) == 23                       # the structure itself, not a copy
    g = N._bind("cap", CAP, ("p", "q"))
    assert g(ctypes.addressof(sp), 16) == 23 and g(None, 16) == -1

    class Tensor:
        def data_ptr(self):
            return ctypes.addressof(sp)
    assert g(Tensor(), 16) == 23


@pytest.mark.parametrize("args,error", [
    ((L.DeltaDesc(), 16), TypeError), ((None, 16), TypeError), ((3, 16), TypeError),
    ((L.DeltaSelectParams(), 1.5), TypeError), ((L.DeltaSelectParams(), 2 ** 31), OverflowError),
    ((L.DeltaSelectParams(), None), TypeError), ((L.DeltaSelectParams(),), TypeError),
    ((L.DeltaSelectParams(), 1, 2), TypeError),
])
def test_wrong_arguments_raise(args, error):
    f = N._bind("cap", CAP, (L.DeltaSelectParams, "i"))
    with pytest.raises(error):
        f(*args)


def test_wrong_pointers_raise():
    g = N._bind("cap", CAP, ("p", "q"))
    with pytest.raises(AttributeError):
        g("text", 16)
    with pytest.raises(OverflowError):
        g(-1, 16)
    with pytest.raises(OverflowError):
        g(2 ** 64, 16)
    with pytest.raises(TypeError):
        N._bind("cap", CAP, ("p", "q"))(None, page_size=16)


def test_bind_refuses_bad_descriptions():
    for kinds in (("x",), ("pi",), (5,), ("p",) * 17):
        with pytest.raises(ValueError):
            N._bind("cap", CAP, kinds)
    with pytest.raises(ValueError):
        N._bind("cap", 0, ("p",))


def test_a_structure_of_the_wrong_type_is_refused_by_the_entry_points():
    with pytest.raises(TypeError):
        L.full_attn_q8(L.DeltaSelectParams(), L.DeltaPageTable(), None, L.DeltaQ8Cache(), None, None, 0)
    with pytest.raises(TypeError):
        L.rope(L.DeltaDesc(), L.DeltaQ8Cache(), 1, None, None, None, None)
