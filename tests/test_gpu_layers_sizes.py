"""The largest sizes that the layers' calls take, and the first that they refuse: more rows than
32 bits hold are not cut down to a few."""
import pytest
import torch

import combine_ep_route_gb300 as ep

pytestmark = pytest.mark.gpu
BF16 = torch.bfloat16


@pytest.fixture(scope="module", autouse=True)
def built():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import __graft_entry__
    __graft_entry__.build()


@pytest.mark.parametrize("rows", [1 << 31, (1 << 32) + 5])
def test_more_rows_than_32_bits_hold_are_refused(rows):
    x = torch.empty(rows, 1, dtype=BF16, device="cuda")
    with pytest.raises(ValueError):
        ep.route_topk(x, 1)
    with pytest.raises(ValueError):
        ep.route_topk_backward(torch.empty(1, 1, device="cuda"), x, torch.empty(1, 1, dtype=torch.int32, device="cuda"))
    x = torch.empty(rows, 8, dtype=BF16, device="cuda")
    with pytest.raises(ValueError):
        ep.linear_wgrad(x, x)
    with pytest.raises(ValueError):
        ep.experts_product_wgrad(x[None], x[None], torch.zeros(1, dtype=torch.int32, device="cuda"))
    with pytest.raises(ValueError):
        ep.linear(x, torch.zeros(8, 8, dtype=BF16, device="cuda"))


def test_the_most_tokens():
    """2^31 - 1 tokens, one expert: all go there, with weight 1 and no gradient."""
    tokens = (1 << 31) - 1
    z = torch.zeros(tokens, 1, dtype=BF16, device="cuda")
    ids = torch.full((tokens, 1), 7, dtype=torch.int32, device="cuda")
    w = torch.full((tokens, 1), 7.0, device="cuda")
    ep.route_topk(z, 1, out=(ids, w))
    assert not ids.any() and (w == 1).all()
    z.fill_(3.0)
    d = torch.full_like(z, 7.0)
    ep.route_topk_backward(w, z, ids, out=d)
    assert not d.any()
