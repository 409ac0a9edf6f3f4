"""The 8-bit cache's kernels where their CTAs go on to a second and third piece
of work, and where one pair's work lies on most of the CTAs: against float64.
Each case is held to the kernels' own division of the work, so that it goes on
reaching the code that it is there for."""
import os
import re

import numpy as np
import pytest

from tests.test_kv8_limits_gpu import _Step

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "rank_transformer_b200", "csrc")


@pytest.fixture(scope="module")
def fs():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from rank_transformer_b200 import flashsvd
    flashsvd.init(0, max_tokens=512, max_rank=512, max_hidden=1024, max_ffn=2048)
    return flashsvd


def _constant(source, name):
    with open(os.path.join(CSRC, source)) as f:
        return int(re.search(r"constexpr int %s = (\d+)" % name, f.read()).group(1))


def _sms():
    return torch.cuda.get_device_properties(0).multi_processor_count


def _attend_split(n, G, rep):
    """(most pairs that one worker has blocks of, most workers of one pair)."""
    cost, least = _constant("kv8_attn.cu", "KA_PAIR_COST"), _constant("kv8_attn.cu", "KA_MIN_UNITS")
    blocks = [x // 64 + 1 for x in n for _ in range(G)]
    total = sum(blocks) + cost * len(blocks)
    workers = min(-(-total // least), _sms() * (2 if rep <= 8 else 1))
    each, more = divmod(total, workers)
    worker_of = lambda u: u // (each + 1) if u < more * (each + 1) else more + (u - more * (each + 1)) // each  # noqa: E731
    pairs, most, at = np.zeros(workers, np.int64), 0, 0
    for b in blocks:
        first, last = worker_of(at), worker_of(at + b - 1)
        pairs[first:last + 1] += 1
        most = max(most, last - first + 1)
        at += b + cost
    return int(pairs.max()), most


@pytest.mark.parametrize("fmt", ["int8", "e4m3"])
@pytest.mark.parametrize("n,G,rep,D,workers", [
    (20000, 1, 1, 64, 128),      # 16 groups of threads share the partials, two batches of loads each
    (65500, 1, 1, 64, 256),
    (65500, 1, 4, 128, 256),
    (33001, 2, 8, 128, 128),
    (20000, 1, 16, 128, 128),
    (16383, 1, 12, 64, 65),
])
def test_attend_joins_many_partials(fs, fmt, n, G, rep, D, workers):
    """A long history of few heads lies on more CTAs than a joining warp keeps
    in registers (64)."""
    assert _attend_split([n], G, rep)[1] >= workers > 64
    s = _Step(fs, fmt, [n], G, rep, D, (n // 64 + 1) * 64, 51, scale=D ** -0.5)
    w = torch.full((1, G, s.S_max), 2.0, device="cuda")
    s.check(s.run(w), w, 2.0)
