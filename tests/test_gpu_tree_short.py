"""bq_tree_accept where a sequence holds fewer tokens than its tree has rows: the length it gives for bq_kv_resize is
never more than the tokens held, so that no token is made of nothing."""
import numpy as np
import pytest

from gpu_helpers import torch_mod
from test_gpu_tree import accept

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    torch = torch_mod()
    if not torch.cuda.is_available():
        pytest.fail("GPU tests need a GPU")
    import bit_quantized_decode_qmv_amd as bq
    bq.load_library()


def test_length_of_a_sequence_shorter_than_its_tree():
    chain = np.arange(-1, 4)                                 # five rows, of which the first four are accepted
    target, token = [1, 2, 3, 9, 9], [0, 1, 2, 3, 4]
    lens = [50, 5, 4, 3, 1, 0, -2]
    path, kept, nxt, want = accept([target] * 7, [token] * 7, [chain] * 7, lens, 8)
    assert kept.tolist() == [4] * 7 and nxt.tolist() == [9] * 7 and (path[:, :5] == [0, 1, 2, 3, -1]).all()
    assert want.tolist() == [49, 4, 4, 3, 1, 0, 0]
