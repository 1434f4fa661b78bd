"""Checks of the paged-cache entry points at the borders of what they accept, without a GPU."""
import pytest

import fourier_basis_attention_b200 as fa
from test_paged_host import rope_args


@pytest.mark.parametrize("kw", [
    dict(xs=(1, 1, 128)), dict(xs=(3, 5, 128), ys=(7, 1, 128)), dict(ys=(-1, 0, 128)),
    dict(xs=(1, 1 << 50, 128), dtype=fa.FA_BF16)], ids=str)
def test_rope_ignores_the_strides_of_axes_of_size_1(kw):
    """H = 0: the checks of the strides pass and nothing is launched."""
    assert fa.LIB.fa_rope(*rope_args(**dict(B=1, T=1, H=0, **kw))) == fa.FA_OK


@pytest.mark.parametrize("axis", range(3))
@pytest.mark.parametrize("stride", [1, -512, 130])
def test_rope_checks_the_strides_of_longer_axes(axis, stride):
    size, strides = [1, 1, 1], [1, 1, 1]
    size[axis], strides[axis] = 2, stride
    kw = dict(zip("BTH", size), xs=tuple(strides), ys=(1 << 20,) * 3)
    assert fa.LIB.fa_rope(*rope_args(**kw)) == fa.FA_ERR_INVALID
    assert f"x_stride[{axis}]" in fa.fa_last_error()
