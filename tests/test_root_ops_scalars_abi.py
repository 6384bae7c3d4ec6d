"""Scalars that are finite as given and not in the fp32 that the kernels compute
in are refused, before anything is launched."""
import pytest

import fsdp_sharded_mixed_flatten_gb300 as zf
from test_root_ops_abi import INVALID, _embed, _embed_grad, _norm, lib  # noqa: F401


@pytest.mark.parametrize("call,over,code", [
    (_embed, dict(scale=1e39), INVALID), (_embed, dict(scale=-1e300), INVALID),
    (_embed_grad, dict(scale=4e38), INVALID), (_norm, dict(eps=1e39), INVALID),
    (_embed, dict(scale=3e38), -4), (_embed_grad, dict(scale=-3e38), -4),
    (_norm, dict(eps=3e38), -4), (_norm, dict(eps=0.0), -4), (_embed, dict(scale=0.0), -4),
])
def test_range_of_scalars(lib, monkeypatch, call, over, code):        # noqa: F811
    monkeypatch.setenv("ZERO_INJECT_FAILURE", "launch")     # nothing runs on a fake address
    assert call(lib, **over) == code, zf.zero_last_error()
