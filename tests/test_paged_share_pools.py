"""What ``vq_paged_copy`` takes as its list of pools."""
import pytest
import torch

from test_paged_share import i32, vq  # noqa: F401  (a fixture)

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("kind", [list, tuple, iter, lambda a: (t for t in a), lambda a: dict(enumerate(a)).values()])
def test_pools_of_any_kind(vq, kind):  # noqa: F811
    pools = [torch.arange(40, device="cuda").reshape(8, 5), torch.arange(24, device="cuda").half().reshape(8, 3)]
    want = [t.clone() for t in pools]
    for t in want:
        t[6] = t[1]
    vq.vq_paged_copy(i32([[1, 6], [-1, -1]]), kind(pools))
    assert all(torch.equal(a, b) for a, b in zip(pools, want))
    with pytest.raises(TypeError, match="pools"):
        vq.vq_paged_copy(i32([[1, 6]]), kind([*pools, None]))
