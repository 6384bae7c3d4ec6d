"""The device status: one read of one word, whichever kernels record in it."""
import math
import os
import subprocess
import sys
import textwrap
import time

import pytest
import torch

import fsdp_sharded_mixed_flatten_gb300 as zf

pytestmark = pytest.mark.gpu

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from fsdp_sharded_mixed_flatten_gb300 import build
    build.build()
    zf.load()


def _best(call, calls=40):
    times = []
    for _ in range(calls):
        t = time.perf_counter()
        call()
        times.append(time.perf_counter() - t)
    return min(times)


def test_the_status_is_one_copy_and_one_synchronisation():
    """It takes as long as reading a tensor's one value (and some Python); three copies, each
    with its own synchronisation, took more than twice as long."""
    word = torch.zeros(1, dtype=torch.int32, device="cuda")
    read, status = (lambda: int(word.cpu())), (lambda: zf.zero_device_status(clear=False))
    for call in (read, status):
        _best(call)
    torch.cuda.synchronize()
    assert any(_best(status) <= 1.6 * _best(read) for _ in range(5))


def test_first_calls_of_a_process_may_be_captured():
    """What a launch looks up once a device is looked up during a capture too."""
    code = """
        import torch, fsdp_sharded_mixed_flatten_gb300 as zf
        zf.load()
        bf = lambda *s: (torch.arange(s[0] * s[-1], device="cuda") % 7 - 3).view(*s).bfloat16()
        n, vocab, d = 40, 500, 128
        h, w, y = bf(n, d), bf(vocab, d), torch.arange(n, device="cuda")
        loss, lse, gl = torch.zeros(n, device="cuda"), torch.zeros(n, device="cuda"), \\
            torch.ones(n, device="cuda")
        dh, dw, out = torch.zeros_like(h), torch.zeros_like(w), torch.zeros_like(h)
        size = max(zf.zero_head_loss_workspace_bytes(n, vocab, d),
                   zf.zero_head_loss_grad_workspace_bytes(n, vocab, d))
        ws = torch.zeros(size, dtype=torch.uint8, device="cuda")
        def calls():
            zf.zero_rms_norm(h, None, None, 1e-5, out)
            zf.zero_head_loss(out, w, y, loss, lse, ws, size)
            zf.zero_head_loss_grad(out, w, y, lse, gl, dh, dw, False, ws, size)
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            calls()
        g.replay()
        torch.cuda.synchronize()
        got = [t.clone() for t in (out, loss, lse, dh, dw)]
        calls()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(got, (out, loss, lse, dh, dw)))
        assert float(dh.float().abs().sum()) > 0 and zf.zero_device_status() == 0
        print("captured")
    """
    p = subprocess.run([sys.executable, "-c", textwrap.dedent(code)], cwd=ROOT, timeout=300,
                       capture_output=True, text=True)
    assert p.returncode == 0 and "captured" in p.stdout, p.stderr[-2000:]


def test_bounded_waits_of_tiles_report_timeout():
    """The wait of the head's products and the norm's rows, when nothing ends it: it runs out,
    is reported, and the context stays usable."""
    assert zf.zero_device_status() == zf.zero.ZERO_DEVICE_OK
    zf.zero_selftest_tile_wait_timeout(20_000_000)          # 20 ms
    assert zf.zero_device_status(clear=False) == zf.zero.ZERO_DEVICE_TIMEOUT
    assert zf.zero_device_status(clear=True) == zf.zero.ZERO_DEVICE_TIMEOUT
    assert zf.zero_device_status() == zf.zero.ZERO_DEVICE_OK
    n, vocab, d = 40, 500, 128
    h = torch.ones((n, d), dtype=torch.bfloat16, device="cuda")
    w = torch.zeros((vocab, d), dtype=torch.bfloat16, device="cuda")
    size = zf.zero_head_loss_workspace_bytes(n, vocab, d)
    loss, ws = torch.empty(n, device="cuda"), torch.empty(size, dtype=torch.uint8, device="cuda")
    zf.zero_rms_norm(h, None, None, 1e-5, h)
    zf.zero_head_loss(h, w, torch.arange(n, device="cuda"), loss, None, ws, size)
    assert float((loss - math.log(vocab)).abs().max()) <= 1e-5
    assert zf.zero_device_status() == zf.zero.ZERO_DEVICE_OK


@pytest.mark.parametrize("limit", [0, -1, 10 ** 9 + 1])
def test_a_limit_out_of_range_is_refused(limit):
    with pytest.raises(zf.ZeroError):
        zf.zero_selftest_tile_wait_timeout(limit)
