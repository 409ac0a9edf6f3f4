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


@pytest.mark.parametrize("fmt", ["int8", None])
def test_everything_runs_on_the_given_stream(fs, fmt):
    """prefill on a side stream leaves nothing behind the work that the current
    stream still has to do; generate gives the same tokens there."""
    prompt = torch.randint(0, 1000, (2, 100), dtype=torch.int32, generator=torch.Generator().manual_seed(4)).pin_memory()
    m = _model(fmt)
    side = torch.cuda.Stream()
    m.capture(side)
    torch.cuda.synchronize()
    with torch.cuda.stream(side):
        want = m.generate(prompt, 9, side)
    side.synchronize()
    lengths = [m.seqlens] + ([m.positions] if fmt else [])
    on_device = prompt.cuda()
    torch.cuda.synchronize()
    for busy in (False, True):  # (once before: first launches and allocations wait for the device)
        m.seqlens.zero_()
        torch.cuda.synchronize()
        if busy:
            torch.cuda._sleep(BUSY)
        m.prefill(on_device, side)
        with torch.cuda.stream(side):
            got = torch.stack(lengths).cpu()   # waits for `side` alone
        assert (got == 100).all()
    assert not torch.cuda.current_stream().query(), "the stream was to be busy"
    tokens = m.generate(prompt, 9, side)
    side.synchronize()
    assert torch.equal(tokens, want)
    torch.cuda.synchronize()
    fs.check_device_status()
    m.release_graphs()
