"""The stream a call runs on when none is given."""
import types

import pytest

torch = pytest.importorskip("torch")


@pytest.fixture(scope="module")
def fs():
    from rank_transformer_b200 import build
    build.build()
    from rank_transformer_b200 import flashsvd
    return flashsvd


def test_without_torch_s_raw_handle(fs, monkeypatch):
    """torch's raw handle is a private function: without it the public call
    gives the stream."""
    monkeypatch.setattr(torch.cuda, "current_stream", lambda: types.SimpleNamespace(cuda_stream=1234))
    for name in ("_cuda_getCurrentRawStream", "_cuda_getDevice"):
        with monkeypatch.context() as m:
            m.delattr(torch._C, name, raising=False)
            assert fs.stream_handle() == 1234
    assert fs.stream_handle(types.SimpleNamespace(cuda_stream=77)) == 77


@pytest.mark.gpu
def test_is_torch_s_current_stream(fs):
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    assert fs.stream_handle() == torch.cuda.current_stream().cuda_stream
    s = torch.cuda.Stream()
    with torch.cuda.stream(s):
        assert fs.stream_handle() == s.cuda_stream
    assert fs.stream_handle(s) == s.cuda_stream
