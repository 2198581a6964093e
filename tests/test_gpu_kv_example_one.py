"""The example decoder with a single sample: nothing to fork."""
import pytest

from test_gpu_kv_example import ex, model, prompt  # noqa: F401

pytestmark = pytest.mark.gpu


def test_one_sample(ex, model):  # noqa: F811
    """The same tokens as the first of two samples gives, whose first token is the same."""
    out = [ex.decode(ex.Session(model, rows=2), prompt(150), samples, 0, 4) for samples in (1, 2)]
    assert out[0][0] == out[1][0][:1]
    session = ex.Session(model, rows=2)
    tokens, logits, moved = ex.decode(session, prompt(150), 1, 3, 4)
    assert len(tokens) == 1 and len(tokens[0]) >= 4 and bool(logits.isfinite().all()) and moved == 0
    # the pages are the sample's, and it holds what was accepted and the last token
    assert int((session.refs > 0).sum()) == -(-int(session.lens[0]) // 64)
    assert int(session.lens[0]) == 150 + len(tokens[0])
