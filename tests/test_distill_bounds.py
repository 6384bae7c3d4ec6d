"""The bounds of distill_bounds.py: finite in rows of any spread, and narrow
enough to notice a planted mistake there.  CPU only."""
import pytest
import torch

import distill_bounds as D
import root_reference as R

F32 = torch.float32


def _rows():
    """Teacher's entries spread over the type's range, in rows of ordinary logits."""
    g = torch.Generator().manual_seed(3)
    n, vocab, top = 5, 300, 8
    z = torch.randn((n, vocab), generator=g) * 3
    ids = (torch.arange(top, dtype=torch.int32) * 11).repeat(n, 1)
    t = torch.randn((n, top), generator=g) * 2
    t[0] = torch.finfo(F32).min
    t[1] = torch.arange(top) * 1e30
    t[2, 1:] = torch.finfo(F32).min
    t[3, 2:] = -1e9
    t[4, 2] = float("-inf")
    w = torch.rand(n, generator=g) + 0.1
    return z, ids, t, w


@pytest.mark.parametrize("tau", [0.5, 1.0])
def test_values_are_those_of_the_definition(tau):
    z, ids, t, w = _rows()
    got, want = D.distill(z, ids, t, w, tau), R.distill(z, ids, t, w, tau)
    torch.testing.assert_close(got["loss"], want["loss"], rtol=1e-12, atol=1e-14)
    torch.testing.assert_close(got["grad"], want["grad"], rtol=1e-12, atol=1e-14)


def test_planted_mistakes_are_noticed():
    """0.1 % off in the largest entry's weight, in its gradient or in the loss,
    in each of the rows."""
    z, ids, t, w = _rows()
    ref = D.distill(z, ids, t, w, 0.5)
    for key, bound in (("loss", "d_loss"), ("grad", "d_grad")):
        assert bool(torch.isfinite(ref[bound]).all())
        D.check(ref[key], ref[key], ref[bound], key)
        for row in range(z.shape[0]):
            wrong = ref[key].clone()
            at = row if key == "loss" else (row, int(ref["grad"][row].abs().argmax()))
            wrong[at] *= 1.001
            with pytest.raises(AssertionError):
                D.check(wrong, ref[key], ref[bound], key)
