"""The 8-bit cache operators at the ends of their ranges: capacities whose
scores do not fit the workspace at once, values near the ends of bf16's range;
against the float64 oracle."""
import math

import numpy as np
import pytest

from oracle import flashsvd_oracle as oracle
from tests.test_kv8_gpu import U32, _attend_bound, _bf16, _dev, _rows

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")


@pytest.fixture(scope="module")
def fs():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from rank_transformer_b200 import flashsvd
    flashsvd.init(0, max_tokens=512, max_rank=512, max_hidden=1024, max_ffn=2048)
    return flashsvd


class _Step:
    """A decode step over rows of n[b] tokens and its comparison with the
    oracle: outputs and, unless None, the weights w added to w0."""

    def __init__(self, fs, fmt, n, G, rep, D, S_max, seed, scale=0.125, vstd=1.0):
        from rank_transformer_b200.kv8 import KV8Cache
        rng = np.random.default_rng(seed)
        B, S = len(n), max(n) + 1
        self.fs, self.n, self.G, self.rep, self.D, self.S_max, self.fmt, self.scale = fs, n, G, rep, D, S_max, fmt, scale
        self.k, self.v = _rows(rng, (B, S, G, D), False), _bf16(vstd * _rows(rng, (B, S, G, D)))
        self.q = _bf16(1.5 * rng.standard_normal((B, G * rep, D)))
        self.cache = KV8Cache(B, G, D, S_max, fmt)
        self.dn = _dev(n, torch.int32)
        fs.kv8_store(_dev(self.k), _dev(self.v), self.cache, self.dn, S, S)
        self.kn = np.stack([self.k[b, n[b]] for b in range(B)])
        self.vn = np.stack([self.v[b, n[b]] for b in range(B)])

    def run(self, w):
        out = torch.full((len(self.n), self.G * self.rep, self.D), 7.0, dtype=torch.bfloat16, device="cuda")
        self.fs.kv8_decode_attn(_dev(self.q), _dev(self.kn), _dev(self.vn), self.cache, self.dn, w, True, out,
                                self.G * self.rep, self.scale)
        torch.cuda.synchronize()
        self.fs.check_device_status()
        return out

    def check(self, out, w, w0):
        got, rep = out.double().cpu().numpy(), self.rep
        for b, n in enumerate(self.n):
            for g in range(self.G):
                kx = oracle.kv8_rows(self.k[b, :n + 1, g], self.fmt)
                vx = oracle.kv8_rows(self.v[b, :n + 1, g], self.fmt)
                add, worst = np.zeros(n + 1), 0.0
                for h in range(g * rep, (g + 1) * rep):
                    p = oracle.attention_probs(self.q[b, h][None], kx, self.scale)[0]
                    want = p @ vx
                    e_out, eps_p = _attend_bound(self.q[b, h], kx, vx, p, self.scale, want)
                    # Below 2^-126 steps are absolute.  Output: bf16's are 2^-133,
                    # half of one 2^-134.  Sums: they carry 2^-shift, 2^(shift - 1)
                    # the least power of two from S_max on, and each of n + 1
                    # additions is off by at most fp32's least step, 2^-149 (matrix
                    # instructions cut off); divided by a sum of probabilities of
                    # 1 or more, that is 2^(shift - 149) each.
                    shift = math.ceil(math.log2(self.S_max)) + 1
                    e_out = e_out + 2.0 ** -134 + (n + 1) * 2.0 ** (shift - 149)
                    err = np.abs(got[b, h] - want)
                    assert np.all(err <= e_out), (b, h, float(np.max(err / e_out)))
                    add += p
                    worst = max(worst, eps_p)
                if w is None:
                    continue
                base = np.full(n + 1, w0)
                base[n] = 0.0     # the appended token's entry is set
                wg = w[b, g, :n + 1].double().cpu().numpy()
                assert np.all(np.abs(wg - base - add) <= worst * add + 4 * U32 * (base + add) + 2.0 ** -100), (b, g)
                assert (w[b, g, n + 1:] == w0).all()


@pytest.mark.parametrize("fmt,n,G,rep,D,S_max,launches", [
    ("int8", [300, 64], 20, 2, 64, 524288, 2 * 2 * 2),    # 16 KV heads' scores fit: 10 and 10 a row
    ("e4m3", [127], 3, 16, 128, 400000, 2 * 2),           # 2 fit: 2 and 1
    ("int8", [70, 0, 5], 2, 8, 64, 1048576, 3 * 2),       # 2 fit: both heads of a row
])
def test_scores_of_a_row_cut_by_heads(fs, fmt, n, G, rep, D, S_max, launches):
    """With weights, the scores of one batch row may pass the workspace: the
    call runs over some of its KV heads at a time."""
    s = _Step(fs, fmt, n, G, rep, D, S_max, 31)
    w = torch.full((len(n), G, S_max), 2.0, device="cuda")
    before = fs.lib.flashsvd_launch_count()
    out = s.run(w)
    assert fs.lib.flashsvd_launch_count() - before == launches
    s.check(out, w, 2.0)


@pytest.mark.parametrize("fmt", ["int8", "e4m3"])
@pytest.mark.parametrize("power", [118, -108])
@pytest.mark.parametrize("n,G,rep,D,S_max", [
    ([4090, 5], 1, 2, 64, 4096),
    ([2047, 64, 0], 2, 1, 128, 2048),
    ([1500], 1, 12, 128, 1536),
    ([63, 190, 128], 3, 9, 64, 192),
])
def test_values_at_the_ends_of_the_range(fmt, power, fs, n, G, rep, D, S_max):
    """Output sums are up to n times the output: values of up to 2^126.5 (and
    down to where the scale of a block is at its floor) give what the
    definition gives, with attention spread over all tokens (scale 2^-6) and
    on a few."""
    for scale in (2.0 ** -6, 0.25):
        s = _Step(fs, fmt, n, G, rep, D, S_max, 41 + D, scale=scale, vstd=2.0 ** power)
        assert np.isfinite(s.v).all() and np.abs(s.v).max() > 2.0 ** (power + 6)
        out = s.run(None)
        assert torch.isfinite(out).all()
        s.check(out, None, 0.0)


def test_a_full_model_refuses_a_step(fs):
    """At capacity a step raises and leaves everything as it was; after an
    eviction it runs."""
    from rank_transformer_b200.model import DecoderConfig, DecoderModel
    cfg = DecoderConfig(layers=2, d=256, H=4, D=64, f=704, vocab=1000, rho=(0.5,))
    m = DecoderModel(cfg, B=2, S_max=128, seed=3, kv_format="int8", kv_keep=70, max_positions=300)
    m.prefill(torch.randint(0, 1000, (2, 127), dtype=torch.int32, device="cuda"))
    m.decode_step_eager()
    torch.cuda.synchronize()
    state = lambda: [t.clone() for c in m.kv8 for t in c.tensors()] + [m.seqlens.clone(), m.kv_weights[1].clone()]  # noqa: E731
    before = state()
    with pytest.raises(ValueError, match="no room"):
        m.decode_step_eager()
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(before, state()))
    m.evict()
    m.decode_step_eager()
    torch.cuda.synchronize()
    fs.check_device_status()
    assert m.length == 71 and m.seqlens.tolist() == [71, 71] and m.positions.tolist() == [129, 129]


@pytest.mark.parametrize("fmt,code", [("int8", 64.0), ("e4m3", 256.0)])
def test_a_code_worth_2_to_128_moves_as_an_infinity(fs, fmt, code):
    """The last bf16 number's code stands for 2^128, which no bf16 row holds:
    the block that it is moved into gets the scale NaN, as with an infinity."""
    from rank_transformer_b200.kv8 import KV8Cache
    n, keep, D = 200, 130, 64
    x = torch.ones((1, n, 1, D), device="cuda").to(torch.bfloat16)
    x[0, 5] = torch.finfo(torch.bfloat16).max
    src, dst = KV8Cache(1, 1, D, 256, fmt), KV8Cache(1, 1, D, 192, fmt)
    fs.kv8_store(x, x, src, None, n, n)
    assert src.k.float()[0, 0, 5, 0] == code and torch.isfinite(src.k_scale).all()
    w = torch.ones((1, 1, 256), device="cuda")
    w[0, 0, 5] = 2.0
    wo, kept = torch.zeros((1, 1, 192), device="cuda"), torch.zeros((1, 1, keep), dtype=torch.int32, device="cuda")
    fs.kv8_evict(src, dst, w, wo, torch.tensor([n], dtype=torch.int32, device="cuda"), None, kept, keep, 0)
    torch.cuda.synchronize()
    fs.check_device_status()
    for s in (dst.k_scale, dst.v_scale):
        assert torch.isnan(s[0, 0, 0]) and s[0, 0, 1] == (2.0 ** -6 if fmt == "int8" else 2.0 ** -8)
    assert not dst.k.float()[0, 0, :64].any()


@pytest.mark.parametrize("fmt", ["int8", "e4m3"])
def test_caches_beyond_32_bits(fs, fmt):
    """The last head's rows lie 2^32 bytes and more behind the first one's:
    stored, attended over, evicted in place and into another cache."""
    from rank_transformer_b200.kv8 import KV8Cache
    from tests.test_kv8_gpu import _check_cache
    n, G, D, S_max, keep = 300, 9, 128, 1 << 22, 130
    s = _Step(fs, fmt, [n], G, 1, D, S_max, 71, scale=D ** -0.5)
    c = s.cache
    assert (G - 1) * S_max * D >= 1 << 32
    w = torch.full((1, G, S_max), 2.0, device="cuda")
    s.check(s.run(w), w, 2.0)
    w[0, :, :n + 1] = torch.rand((G, n + 1), generator=torch.Generator("cuda").manual_seed(5), device="cuda")
    wh = w[0, :, :n + 1].double().cpu().numpy()
    seq = torch.tensor([n + 1], dtype=torch.int32, device="cuda")
    kept = torch.zeros((1, G, keep), dtype=torch.int32, device="cuda")
    small = KV8Cache(1, G, D, 192, fmt)
    for dst, wo in ((small, torch.zeros((1, G, 192), device="cuda")), (c, w)):
        fs.kv8_evict(c, dst, w, wo, seq, None, kept, keep, 20)
        torch.cuda.synchronize()
        fs.check_device_status()
        host = [dict(codes=a[:, :, :192].float().cpu().double().numpy(), scale=x[:, :, :3].cpu().double().numpy(),
                     tail=t.cpu().double().numpy()) for a, x, t in ((dst.k, dst.k_scale, dst.k_tail),
                                                                   (dst.v, dst.v_scale, dst.v_tail))]
        for g in range(G):
            idx = oracle.evict_kept(wh[g], keep, 20)
            assert kept[0, g].tolist() == idx.tolist()
            np.testing.assert_array_equal(wo[0, g, :keep].double().cpu().numpy(), wh[g][idx])
            for i, rows in enumerate((s.k, s.v)):
                held = oracle.kv8_rows(rows[0, :, g], fmt)[idx]
                if dst is small:
                    old = [{k: np.zeros_like(v) for k, v in h.items()} for h in host]
                else:     # what lies behind the kept rows stays
                    old = [{k: v.copy() for k, v in h.items()} for h in host]
                _check_cache(host, old, i, 0, g, held, fmt)


def test_weight_sums_beyond_32_bits(fs):
    """The window's queries and the last keys lie beyond 2^32 bytes."""
    S, H, D, window = 70000, 256, 128, 64
    assert (S - window) * H * D * 2 > 1 << 32
    g = torch.Generator("cuda").manual_seed(9)
    q, k = (torch.empty((1, S, H, D), dtype=torch.bfloat16, device="cuda").normal_(generator=g) for _ in range(2))
    w = torch.zeros((1, H, S), device="cuda")
    fs.attn_weight_sums(q, k, w, None, 1, S, H, H, D, S, S, window, D ** -0.5)
    torch.cuda.synchronize()
    fs.check_device_status()
    hidden = torch.arange(S, device="cuda")[None, :] > torch.arange(S - window, S, device="cuda")[:, None]
    for h in (0, 1, 100, 254, 255):
        qd, kd = q[0, S - window:, h].double(), k[0, :, h].double()
        want = torch.softmax((qd @ kd.T * D ** -0.5).masked_fill(hidden, -float("inf")), -1).sum(0)
        # the bound of test_kv8_gpu._sums_bound
        d = D ** -0.5 * float((qd.abs() @ kd.abs().amax(0)).max()) * (D + 24) * 2 * U32
        bound = want * (2 * d + 2.0 ** -19 + (S / 4 + 64) * 2 * U32) + 1e-30
        err = (w[0, h].double() - want).abs()
        assert (err <= bound).all(), (h, float((err / bound).max()))
