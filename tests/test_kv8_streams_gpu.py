"""The model over 8-bit caches on a stream that is not torch's current one."""
import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")

BUSY = 400_000_000  # clocks: a fifth of a second


@pytest.fixture(scope="module")
def fs():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from rank_transformer_b200 import flashsvd
    flashsvd.init(0, max_tokens=1024, max_rank=512, max_hidden=1024, max_ffn=2048)
    return flashsvd


def _model(fmt, **kw):
    from rank_transformer_b200.model import DecoderConfig, DecoderModel
    cfg = DecoderConfig(layers=2, d=256, H=4, D=64, f=704, vocab=1000, rho=(0.5,))
    return DecoderModel(cfg, B=2, S_max=192, seed=3, kv_format=fmt, **kw)


def test_replaced_prompt_scratch_is_not_handed_out(fs):
    """A buffer that a busy stream uses goes back to the allocator only when
    that stream is done with it, whichever stream replaces it."""
    m = _model("int8")
    side = torch.cuda.Stream()
    for first, second in ((side, None), (None, side)):
        with torch.cuda.stream(first):
            m._prompt_rows(300)
        torch.cuda.synchronize()
        with torch.cuda.stream(side):
            torch.cuda._sleep(BUSY)
            old = m._prompt_rows(300)
            old.zero_()
        at = old.data_ptr()
        del old
        with torch.cuda.stream(second):
            m._prompt_rows(301)
        free = [torch.empty((2, 300, 256), dtype=torch.bfloat16, device="cuda") for _ in range(4)]
        assert not side.query(), "the stream was to be busy"
        assert at not in [t.data_ptr() for t in free]
        torch.cuda.synchronize()
