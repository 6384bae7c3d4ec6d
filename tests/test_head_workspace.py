"""What the head's cross entropy asks for as a workspace: a workspace for a batch does for
every shorter one."""
import random

import pytest

import fsdp_sharded_mixed_flatten_gb300 as zf

QUERIES = [zf.zero_head_loss_workspace_bytes, zf.zero_head_loss_grad_workspace_bytes]
SIZE = -3


@pytest.fixture(scope="module", autouse=True)
def _built():
    from fsdp_sharded_mixed_flatten_gb300 import build
    build.build()


@pytest.mark.parametrize("query", QUERIES)
@pytest.mark.parametrize("vocab,dim", [(131072, 4096), (131072, 768), (50257, 768), (1000, 64),
                                       (32003, 770), (128256, 8192), (300, 4000)])
def test_needs_grow_with_the_tokens(query, vocab, dim):
    rng = random.Random(vocab + dim)
    sizes = sorted({1, 2, 31, 32, 33, 63, 64, 65, 127, 128, 129, 255, 256, 257, 512, 513, 1000,
                    1024, 2048, 3000, 4096, 8192, 8193, 16384, 20000}
                   | {rng.randrange(1, 20000) for _ in range(20)})
    needs = [query(n, vocab, dim) for n in sizes]
    assert needs == sorted(needs), [(n, b) for n, b in zip(sizes, needs)]


@pytest.mark.parametrize("vocab,dim,longest", [(131072, 4096, 8192), (131072, 768, 16384),
                                               (50257, 768, 8192), (32003, 770, 4096)])
def test_a_workspace_for_the_longest_batch_is_enough(vocab, dim, longest):
    """Calls with fake addresses: none is refused for its workspace.  (Without a device the
    launch behind the checks fails; where there is one, nothing is launched here.)"""
    import torch
    if torch.cuda.is_available():
        pytest.skip("fake addresses never reach a GPU")
    lib = zf.load()
    at = [0x100000 * (i + 1) for i in range(8)]
    loss, grad = (q(longest, vocab, dim) for q in QUERIES)
    for n in [1, 33, 64, 65, 200, 256, 257, 1000, 2048, 4096, longest - 1, longest]:
        for table in (at[1], at[1] + 2):
            rc = lib.zero_head_loss(at[0], n, dim, dim, table, vocab, at[2], 8, at[3], at[4], at[5],
                                    loss, None)
            assert rc != SIZE, zf.zero_last_error()
            rc = lib.zero_head_loss_grad(at[0], n, dim, dim, table, vocab, at[2], 8, at[4], at[3],
                                         at[6], dim, at[7], 0, at[5], grad, None)
            assert rc != SIZE, zf.zero_last_error()


def test_queries_of_the_most_tokens_answer():
    for query in QUERIES:
        assert query(zf.ZERO_MAX_HEAD_TOKENS, 1000, 64) > 0


IN_PLACE = [zf.zero_head_loss_in_place_workspace_bytes,
            zf.zero_head_loss_grad_in_place_workspace_bytes]


@pytest.mark.parametrize("n,vocab,dim", [(1, 131072, 4096), (32, 131072, 4096),
                                         (128, 128000, 4096), (8192, 131072, 4096),
                                         (1, 128256, 8192), (1024, 32000, 768)])
def test_a_table_read_in_place_needs_no_copy(n, vocab, dim):
    """The gradient's copies of the tokens' rows, its dz (at most 512 MB) and its sums (at most
    512 MB, or one part of them) in whole tiles of 256 tokens; nothing of the table's size."""
    rows = (n + 255) // 256 * 256
    loss, grad = (q(n, vocab, dim) for q in IN_PLACE)
    small = 16 * 1024 + 16 * n
    dz = min(2 * rows * (vocab + 255), 512 << 20)
    sums = max(min(64 * 4 * rows * dim, 512 << 20), 4 * rows * dim)
    assert loss <= 2 * rows * dim + 8 * n * (vocab // 32 + 1 + 1024) + 2 * small
    assert grad <= 2 * rows * dim + dz + sums + 2 * small
    for q, any_place in zip(IN_PLACE, QUERIES):
        assert q(n, vocab, dim) <= any_place(n, vocab, dim)
        needs = [q(m, vocab, dim) for m in (1, 64, 65, 300, 1000, 5000)]
        assert needs == sorted(needs)


def test_a_call_needs_what_its_own_table_needs():
    """Fake addresses, as above: what is enough in place is refused off the 16-byte grid."""
    import torch
    if torch.cuda.is_available():
        pytest.skip("fake addresses never reach a GPU")
    lib = zf.load()
    at = [0x100000 * (i + 1) for i in range(8)]
    n, vocab, dim = 32, 131072, 4096
    grad = IN_PLACE[1](n, vocab, dim)
    call = lambda table: lib.zero_head_loss_grad(                # noqa: E731
        at[0], n, dim, dim, table, vocab, at[2], 8, at[4], at[3], at[6], dim, at[7], 0, at[5], grad,
        None)
    assert call(at[1]) != SIZE and call(at[1] + 2) == SIZE


def test_a_width_that_is_never_read_in_place_is_refused():
    for query in IN_PLACE:
        with pytest.raises(zf.ZeroError):
            query(10, 100, 12)
