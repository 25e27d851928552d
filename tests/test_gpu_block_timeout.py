"""The bounded-wait failure path of the tensor-core block-attention kernels, run on purpose.

Every wait in them has a limit.  With gattn_block_set_wait_test the computing warps treat their
first wait as expired and leave, so every other warp of the CTA runs into its own limit,
waits for the copies and products that it has in flight, and returns.  No wait is without
an end.  The tests check that the kernels report the timeout, that the record is cleared, and that
the next calls are right.
"""
import pytest

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():
    pytest.skip("needs a CUDA GPU", allow_module_level=True)

pytestmark = pytest.mark.gpu

from gnn_sparse_attention_gb300 import binding as gb  # noqa: E402

TIMEOUT, DEV = 6, "cuda"


def _expect_timeout():
    with pytest.raises(gb.GattnError) as e:
        gb.gattn_block_check_errors()
    assert e.value.status == TIMEOUT
    gb.gattn_block_check_errors()  # the record was cleared


# D, query heads, key heads, q_block: single tiles and pairs of them at both widths, single tokens
CASES = [(64, 2, 2, 128), (64, 16, 4, 128), (128, 2, 2, 64), (128, 16, 4, 128), (128, 8, 2, 1)]


@pytest.mark.parametrize("D,H,Hkv,qb", CASES)
def test_block_wait_timeout_is_reported_and_the_next_call_is_right(D, H, Hkv, qb):
    N = 2500 if qb > 1 else 5
    keys, block, topk = 2500, 64, 12
    g = torch.Generator(device=DEV).manual_seed(3)
    Q, G = (torch.randn(N, H, D, generator=g, device=DEV).to(torch.bfloat16) for _ in range(2))
    K, V = (torch.randn(keys, Hkv, D, generator=g, device=DEV).to(torch.bfloat16) for _ in range(2))
    sq, sk = (torch.tensor([0, n], dtype=torch.int32, device=DEV) for n in (N, keys))
    idx = gb.gattn_block_select(Q, gb.gattn_block_sums(K, sk, block), sq, sk, topk, block, qb, keys)

    def both():
        o, l = gb.gattn_block_fwd(Q, K, V, idx, sq, sk, block, qb)
        return o, l, *gb.gattn_block_bwd(Q, K, V, idx, sq, sk, o, G, l, block, qb)

    want = both()
    gb.gattn_block_check_errors()
    try:
        gb.gattn_block_set_wait_test(True)
        gb.gattn_block_fwd(Q, K, V, idx, sq, sk, block, qb)
        _expect_timeout()
        gb.gattn_block_bwd(Q, K, V, idx, sq, sk, want[0], G, want[1], block, qb)
        _expect_timeout()
    finally:
        gb.gattn_block_set_wait_test(False)
    assert float(torch.ones(1 << 20, device=DEV).sum()) == float(1 << 20)
    for _ in range(2):
        assert all(torch.equal(a, b) for a, b in zip(want, both()))
    gb.gattn_block_check_errors()
