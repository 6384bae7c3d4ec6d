"""In-place calls of the operators around the root unit: rows that share a
start and not a stride would overwrite one another's inputs, and are refused
before anything is launched.  Fake addresses, never dereferenced."""
import pytest

import fsdp_sharded_mixed_flatten_gb300 as zf
from test_root_ops_abi import A, SIZE, _distill, _norm, _norm_grad, lib  # noqa: F401


@pytest.mark.parametrize("call,over", [
    (_norm, dict(out=A[0], os=24)), (_norm, dict(out=A[0], xs=32)),
    (_norm_grad, dict(dx=A[0], dxs=24)), (_norm_grad, dict(dx=A[1], dxs=24)),
    (_norm_grad, dict(dx=A[1], xs=17)), (_distill, dict(dz=A[0], ds=104)),
])
def test_in_place_with_another_stride_is_refused(lib, monkeypatch, call, over):  # noqa: F811
    monkeypatch.setenv("ZERO_INJECT_FAILURE", "launch")     # nothing runs on a fake address
    assert call(lib, **over) == SIZE
    assert "same row stride" in zf.zero_last_error()


@pytest.mark.parametrize("call,over", [
    (_norm, dict(out=A[0])), (_norm_grad, dict(dx=A[0])), (_norm_grad, dict(dx=A[1])),
    (_distill, dict(dz=A[0])),
    # one row: its stride is of no account
    (_norm, dict(out=A[0], os=24, n=1)), (_norm_grad, dict(dx=A[0], dxs=24, n=1)),
    (_distill, dict(dz=A[0], ds=104, n=1)),
])
def test_in_place_that_fits_is_taken(lib, monkeypatch, call, over):   # noqa: F811
    """As far as the launch, which is not made."""
    monkeypatch.setenv("ZERO_INJECT_FAILURE", "launch")
    assert call(lib, **over) == -4
    assert "injected failure" in zf.zero_last_error()
