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
    m.__dict__.update({**dict(kv_format="int8", kv_keep=None, S_max=128, max_positions=200, length=0, position=0), **kw})
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


def _unit(t):
    return t.numel() * t.element_size()


@pytest.mark.parametrize("context", [0, 5, 64, 200])
def test_step_bytes(model, context):
    """Both byte counts hold the same cache traffic, that of the tensors."""
    import torch
    from rank_transformer_b200.kv8 import KV8Cache
    cfg = model.DecoderConfig(layers=3, d=256, H=4, D=64, f=704, vocab=100)
    w = {"U": torch.zeros((16, 8), dtype=torch.bfloat16)}
    head = torch.zeros((256, 100), dtype=torch.bfloat16)

    def counts(**kw):
        m = _model(model, cfg=cfg, B=2, layers=[w], W_lm=head, **{"kv_format": "int8", "kv_keep": None, **kw})
        act = 2 * 256 * 2 * 2 * 3
        step, layers = m.decode_step_bytes(context), m.layers_decode_bytes(context)
        assert step - layers == _unit(head)
        return layers - act - _unit(w["U"])

    assert counts(kv_format=None) == 3 * 2 * 2 * (context + 1) * 256 * 2
    full = context // 64
    c = KV8Cache(2, 4, 64, 64 * max(full, 1), device="cpu")
    history = (_unit(c.k) + _unit(c.k_scale)) * 2 if full else 0
    tail = 2 * _unit(c.k_tail) // 64 * (context % 64 + 1)
    assert counts() == counts(kv_format="e4m3") == 3 * (history + tail)
    weights = 3 * 2 * 4 * (8 * context + 4)    # read and written, the new token's written
    assert counts(kv_keep=32) == 3 * (history + tail) + weights
