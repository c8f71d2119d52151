"""What the norm, the paged cache and attention over it do at their edges, for
instance with values that are not finite where a kernel could lose or spread them.

Tolerances as in test_tree_gpu.py, where nothing else is said.
"""
import pytest

torch = pytest.importorskip("torch")

import io_aware_exact_06_gb300 as fa
from tests import serve_ref as ref
from tests.test_cache_gpu import make, normal, put
from tests.test_tree_gpu import call

pytestmark = pytest.mark.gpu

ROWS = [1, 2, 3, 24, 40]  # query heads to a key head: 6, 12, 18, 144 and 240 rows with six new tokens
NAN, INF = float("nan"), float("inf")


@pytest.fixture(scope="module")
def dev():
    import __graft_entry__
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    __graft_entry__.build()
    return torch.device("cuda:0")


@pytest.mark.parametrize("G", ROWS)
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("codes", [False, True])
@pytest.mark.parametrize("spot,large", [(5, 200), (200, 5), (5, 300), (300, 130)])
def test_nan_keys_beside_large_scores(dev, codes, d, G, spot, large):
    """A NaN key that every row sees makes every row NaN, however far the scores of
    other key tiles lie above it (here more than 2^126 in weight) and whichever tile
    holds it.  One piece a segment, so that tiles meet inside the launch."""
    L, ns, H = 400, [6], 1
    c = make(dev, 600, [L], H, d, 16, codes)
    kv = normal(dev, 601, L, 2, d)
    kv[large, 0] = 160.0 / d ** 0.5  # score about 160 against a query of ones
    put(dev, c, kv[:, :1], kv[:, 1:], [L], [L])
    row = int(ref.row_index(c["page_table"].cpu(), 16, 0, torch.tensor(spot)))
    if codes:
        c["k_cache"].view(torch.uint8)[row // 16, row % 16, :, 3] = 0x7f
    else:
        c["k_cache"][row // 16, row % 16, :, 3] = NAN
    q = torch.ones(6, H * G, d, dtype=torch.bfloat16, device=dev)
    o, lse = call(dev, c, q, [L], ns, None, num_splits=1)
    assert fa.attn_last_device_error() == 0
    assert o.isnan().all() and lse.isnan().all()


@pytest.mark.parametrize("G", ROWS)
@pytest.mark.parametrize("codes", [False, True])
@pytest.mark.parametrize("spot,large", [(5, 200), (200, 5)])
def test_infinite_values_beside_large_scores(dev, codes, G, spot, large):
    """An infinite or NaN value of the context with next to no weight: its channel is not finite."""
    L, ns, H, d = 400, [6], 1, 128
    c = make(dev, 605, [L], H, d, 16, codes)
    kv = normal(dev, 606, L, 2, d)
    kv[large, 0] = 160.0 / d ** 0.5
    put(dev, c, kv[:, :1], kv[:, 1:], [L], [L])
    row = int(ref.row_index(c["page_table"].cpu(), 16, 0, torch.tensor(spot)))
    if codes:
        c["v_cache"].view(torch.uint8)[row // 16, row % 16, :, 3] = 0x7f
    else:
        c["v_cache"][row // 16, row % 16, :, 3] = INF
    q = torch.ones(6, H * G, d, dtype=torch.bfloat16, device=dev)
    o, lse = call(dev, c, q, [L], ns, None, num_splits=1)
    assert fa.attn_last_device_error() == 0
    assert not o[..., 3].isfinite().any() and lse.isfinite().all()
    assert o[..., :3].isfinite().all() and o[..., 4:].isfinite().all()
