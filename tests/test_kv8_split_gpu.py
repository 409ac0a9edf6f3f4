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


@pytest.mark.parametrize("fmt", ["int8", "e4m3"])
@pytest.mark.parametrize("B,G,rep,D,longest,pairs", [
    (48, 8, 2, 64, 200, 2),
    (48, 8, 9, 64, 200, 3),
    (32, 32, 1, 128, 130, 3),
    (40, 5, 16, 128, 300, 2),
    (64, 16, 1, 64, 0, 3),
])
def test_attend_workers_go_on_to_other_pairs(fs, fmt, B, G, rep, D, longest, pairs):
    """Many short histories: a worker has the end of one pair, whole ones, and
    the beginning of another, and may join two."""
    n = [(longest * (7 * b % B)) // (B - 1) for b in range(B)]
    assert _attend_split(n, G, rep)[0] >= pairs
    s = _Step(fs, fmt, n, G, rep, D, 320, 61, scale=D ** -0.5)
    w = torch.full((B, G, 320), 2.0, device="cuda")
    s.check(s.run(w), w, 2.0)


def _sums_items(B, S, G, rep, window):
    """Items of the two launches of the weight sums."""
    runs = -(-min(window, S) // 64)
    tiles = B * G * -(-runs * rep // 2)
    parts = -(-2 * -(-S // 128) // _constant("attn_sums.cu", "SU_MIN_TILES"))
    return tiles * max(1, min(2 * _sms() // tiles, parts)), B * G * -(-S // 128)


@pytest.mark.parametrize("B,S,G,rep,D,window,lens", [
    (8, 1300, 8, 1, 64, 1300, [1300, 0, 700, 1, 1299, 130, 1300, 64]),
    (8, 1300, 8, 1, 128, 1300, [1, 1300, 1300, 0, 65, 1281, 900, 1300]),
    (16, 1290, 8, 5, 64, 100, [1290 - 83 * b for b in range(15)] + [0]),
    (16, 1290, 8, 5, 128, 100, [1, 0] + [1290] * 6 + [129, 1, 0, 1000, 40, 1289, 200, 1290]),
    (20, 400, 16, 3, 64, 170, None),
])
def test_weight_sums_in_several_rounds(fs, B, S, G, rep, D, window, lens):
    """More than two items a resident CTA in both launches: each CTA carries
    its ring, buffers and barrier phases from item to item, passing over items
    of rows that have ended."""
    from tests.test_kv8_gpu import U32
    assert min(_sums_items(B, S, G, rep, window)) > 2 * 2 * _sms()
    g = torch.Generator("cuda").manual_seed(S + D)
    H, scale = G * rep, D ** -0.5
    q = (1.5 * torch.randn((B, S, H, D), generator=g, device="cuda")).to(torch.bfloat16)
    k = torch.randn((B, S, G, D), generator=g, device="cuda").to(torch.bfloat16)
    n = lens or [S] * B
    for b in range(B):
        q[b, n[b]:], k[b, n[b]:] = float("nan"), float("inf")
    w = torch.full((B, G, S), 7.0, device="cuda")
    dl = None if lens is None else torch.tensor(lens, dtype=torch.int32, device="cuda")
    fs.attn_weight_sums(q, k, w, dl, B, S, H, G, D, S, S, window, scale)
    torch.cuda.synchronize()
    fs.check_device_status()
    for b in range(B):
        assert (w[b, :, n[b]:] == 7.0).all()
        if n[b] == 0:
            continue
        lo = max(0, n[b] - window)
        qd = q[b, lo:n[b]].double().view(n[b] - lo, G, rep, D).permute(1, 2, 0, 3)      # [G, rep, W, D]
        kd = k[b, :n[b]].double().permute(1, 0, 2)[:, None]                             # [G, 1, n, D]
        x = qd @ kd.transpose(2, 3) * scale
        hidden = torch.arange(n[b], device="cuda")[None, :] > torch.arange(lo, n[b], device="cuda")[:, None]
        want = torch.softmax(x.masked_fill(hidden, -float("inf")), -1).sum((1, 2))      # [G, n]
        # the bound of test_kv8_gpu._sums_bound, for the largest query of all heads
        d = scale * float((qd.abs() @ kd.abs().amax(2, keepdim=True).transpose(2, 3)).max()) * (D + 24) * 2 * U32
        bound = want * (2 * d + 2.0 ** -19 + (n[b] / 4 + 64) * 2 * U32) + 1e-30
        err = (w[b, :, :n[b]].double() - want).abs()
        assert (err <= bound).all(), (b, float((err / bound).max()))
