"""The tree-verification operators on the GPU: the forms, sizes and calls that only a served batch or a long cache reaches."""
import pytest
import torch

from test_gpu_verify import check_attention, q  # noqa: F401  (q is a fixture)
from verify_helpers import DTYPES, Trees, gen, random_tree

pytestmark = pytest.mark.gpu


# ----------------------------------------------------------------- attention

@pytest.mark.parametrize("dim,page", [(64, 256), (128, 64), (256, 16)])
@pytest.mark.parametrize("more", [1, 64, 130])
def test_attention_many_laps_of_the_ring(q, dim, page, more):
    """Every CTA's run goes around the ring of tiles several times before the tiles that need care."""
    rows = 148 * 20 * (64 if dim == 256 else 128)
    check_attention(q, Trees([rows + more], [[-1, 0, 0]], 2, 1, dim, page, DTYPES["bf16"], seed=more))
