"""How many clusters the table gradient's sort launch takes, on GPUs of any size:
compiled from the plan's own source.  CPU only."""
import ctypes
import os
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
CSRC = os.path.join(ROOT, "fsdp_sharded_mixed_flatten_gb300", "csrc")


@pytest.fixture(scope="module")
def clusters(tmp_path_factory):
    d = tmp_path_factory.mktemp("plan")
    src, lib = str(d / "plan.cc"), str(d / "plan.so")
    with open(src, "w") as f:
        f.write('#include "zero_plan.cuh"\n'
                'extern "C" int clusters(long long vocab, int accumulate, int sms) '
                '{ return zf::sort_clusters(vocab, accumulate != 0, sms); }\n')
    subprocess.run(["g++", "-std=c++17", "-shared", "-fPIC", "-I", CSRC, src, "-o", lib], check=True)
    fn = ctypes.CDLL(lib).clusters
    fn.argtypes = [ctypes.c_longlong, ctypes.c_int, ctypes.c_int]
    return fn


@pytest.mark.parametrize("sms", [1, 2, 3, 4, 7, 8, 16, 78, 152])
@pytest.mark.parametrize("vocab", [1, 31, 257, 50257, 131072, 2 ** 31 - 2])
def test_some_cluster_writes_the_zeros(clusters, vocab, sms):
    assert clusters(vocab, 1, sms) == 1                    # the sort alone
    n = clusters(vocab, 0, sms)
    assert n >= 2                                          # the sort, and one for the zeros
    assert n == 2 or (n - 1) * 8 <= 2 * sms - 8            # no more than the GPU holds
    assert n == 2 or (n - 2) * 8 * 32 < vocab              # nor than there are rows for


def test_of_152_sms(clusters):
    assert clusters(50257, 0, 152) == 38 and clusters(300, 0, 152) == 3
