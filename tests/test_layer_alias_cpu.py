"""In-place uses of the residual norm: an output may be the very buffer of one
input, and of another input only if that has the same rows.  Fake addresses, as
in test_layer_abi_cpu.py."""
import pytest

from causal_linear_attention_fwd_b200 import _binding as B
from test_layer_abi_cpu import DG, DU, DY, H, HN, INV, N, Y, lib, no_gpu, residual, residual_back  # noqa: F401

MIXED = dict(hd=B.LA2_F32, dt=B.LA2_BF16)
SAME = dict(hd=B.LA2_BF16, dt=B.LA2_BF16)


def test_rows_of_unlike_types_on_one_place_are_refused(lib):  # noqa: F811
    """h fp32 and y bf16 from one address: row t of one lies on rows 2 t and 2 t +
    1 of the other, so an output over either meets rows not yet read."""
    assert residual(lib, h=H, y=H, hn=H, n=N, **MIXED) == INV
    assert residual(lib, h=H, y=H, hn=HN, n=H, **MIXED) == INV
    # the gradient of n and of h' from one address, dh over both
    assert residual_back(lib, dn=DG, dhn=DG, dh=DG, **MIXED) == INV


@no_gpu
@pytest.mark.parametrize("types", [SAME, dict(hd=B.LA2_F32, dt=B.LA2_F32)])
def test_rows_of_one_type_on_one_place_pass(lib, types):  # noqa: F811
    """The same rows twice: each is read before it is written."""
    assert residual(lib, h=H, y=H, hn=H, n=N, **types) == B.LA2_ERR_CUDA
    assert residual(lib, h=H, y=H, hn=HN, n=H, **types) == B.LA2_ERR_CUDA
    assert residual_back(lib, dn=DG, dhn=DG, dh=DG, dy=DY, **types) == B.LA2_ERR_CUDA
    assert residual(lib, h=H, y=Y, hn=H, n=Y, **types) == B.LA2_ERR_CUDA
    assert residual_back(lib, dn=DU, dhn=DG, dh=DG, **types) == B.LA2_ERR_CUDA
