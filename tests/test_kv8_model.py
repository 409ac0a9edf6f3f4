"""Host logic of the model over 8-bit caches (no GPU)."""
import types

import pytest

pytest.importorskip("torch")


@pytest.fixture(scope="module")
def model():
    from rank_transformer_b200 import build
    build.build()
    from rank_transformer_b200 import model as m
    return m


def _model(model, **kw):
    """A model's host state, without its tensors."""
    m = model.DecoderModel.__new__(model.DecoderModel)
    m.__dict__.update(dict(kv_format="int8", kv_keep=None, S_max=128, max_positions=200, length=0, position=0,
                           graphs=None, seqlens=None), **kw)
    return m


@pytest.mark.parametrize("length,position", [(128, 128), (60, 200), (128, 200)])
def test_no_step_without_room(model, length, position):
    """A full cache, or a position behind the rotary tables: nothing runs."""
    ran = []
    m = _model(model, length=length, position=position, cfg=None,
               step_graph=types.SimpleNamespace(replay=ran.append))
    for step in (m.decode_step, m.decode_step_eager):
        with pytest.raises(ValueError, match="no room"):
            step()
    assert not ran and (m.length, m.position) == (length, position)
    m.length, m.position = 127, 199
    m.decode_step()
    assert len(ran) == 1 and (m.length, m.position) == (128, 200)
    with pytest.raises(ValueError):
        m.decode_step()
    m.kv_format = None      # the bf16 model goes by its device lengths alone
    m.decode_step()
    assert len(ran) == 2
