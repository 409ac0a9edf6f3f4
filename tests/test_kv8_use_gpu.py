"""The 8-bit cache operators as a server uses them: two contexts at once,
captured graphs that share a workspace, batches cut by the workspace, and the
refusals that need an initialised library.  Everything here is compared bit
for bit: the operators have no atomics in their sums, so equal inputs and an
equal work split give equal results."""
import threading

import numpy as np
import pytest

from oracle import flashsvd_oracle as oracle

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")

INVALID, MISALIGNED, UNSUPPORTED = 1, 2, 3


@pytest.fixture(scope="module")
def fs():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from rank_transformer_b200 import flashsvd
    flashsvd.init(0, max_tokens=512, max_rank=512, max_hidden=1024, max_ffn=2048)
    return flashsvd


def _normal(seed, *shape):
    g = torch.Generator("cuda").manual_seed(seed)
    return torch.randn(shape, generator=g, device="cuda").to(torch.bfloat16)


class _Chain:
    """A prompt of S tokens with the weights of its last `window` queries,
    `steps` decode steps, an eviction in place to `keep`, `steps` more."""

    def __init__(self, fs, seed, B, G, rep, D, S_max, S, window, steps, keep, recent, fmt):
        from rank_transformer_b200.kv8 import KV8Cache
        self.fs, self.dims, self.keep, self.recent = fs, (B, G, rep, D, S_max, S, window), keep, recent
        self.k, self.v = _normal(seed, B, S, G, D), _normal(seed + 1, B, S, G, D)
        self.q = _normal(seed + 2, B, S, G * rep, D)
        self.lens = torch.tensor([S - 37 * b for b in range(B)], dtype=torch.int32, device="cuda")
        self.kn, self.vn = _normal(seed + 3, 2 * steps, B, G, D), _normal(seed + 4, 2 * steps, B, G, D)
        self.qn = _normal(seed + 5, 2 * steps, B, G * rep, D)
        self.cache = KV8Cache(B, G, D, S_max, fmt)
        self.weights = torch.zeros((B, G, S_max), device="cuda")
        self.n = torch.zeros(B, dtype=torch.int32, device="cuda")
        self.kept = torch.zeros((B, G, keep), dtype=torch.int32, device="cuda")
        self.out = torch.zeros((2 * steps, B, G * rep, D), dtype=torch.bfloat16, device="cuda")
        self.steps = steps

    def reset(self):
        for t in (*self.cache.tensors(), self.weights, self.kept, self.out):
            t.view(torch.uint8).zero_()
        self.n.copy_(self.lens)

    def run(self, stream=None):
        fs, c = self.fs, self.cache
        B, G, rep, D, S_max, S, window = self.dims
        fs.kv8_store(self.k, self.v, c, self.lens, S, S, stream)
        fs.attn_weight_sums(self.q, self.k, self.weights, self.lens, B, S, G * rep, G, D, S, S_max, window,
                            D ** -0.5, stream)
        for t in range(2 * self.steps):
            if t == self.steps:
                fs.kv8_evict(c, c, self.weights, self.weights, self.n, self.n, self.kept, self.keep, self.recent,
                             stream)
            fs.kv8_decode_attn(self.qn[t], self.kn[t], self.vn[t], c, self.n, self.weights, True, self.out[t],
                               G * rep, D ** -0.5, stream)
            fs.advance_seqlens(self.n, B, stream)

    def state(self):
        return [t.clone() for t in (*(x.view(torch.uint8) for x in self.cache.tensors()), self.weights, self.n,
                                    self.kept, self.out)]

    def eager(self):
        self.reset()
        self.run()
        torch.cuda.synchronize()
        self.fs.check_device_status()
        assert torch.equal(self.n, torch.minimum(self.lens + self.steps, torch.full_like(self.n, self.keep))
                           + self.steps)
        return self.state()


def _same(a, b):
    return all(torch.equal(x, y) for x, y in zip(a, b))


def _chains(fs):
    return [_Chain(fs, 10, 2, 3, 2, 64, 512, 400, 100, 7, 130, 20, "int8"),
            _Chain(fs, 50, 3, 2, 8, 128, 1088, 1030, 1030, 5, 700, 0, "e4m3")]


def test_two_contexts_two_streams_concurrently(fs):
    """Two host threads, each with its own context, stream and chain, give
    what the default context gives for one after the other."""
    chains = _chains(fs)
    want = [c.eager() for c in chains]
    ctxs = [fs.Context(0, max_tokens=512, max_rank=512, max_hidden=1024, max_ffn=2048) for _ in chains]
    streams = [torch.cuda.Stream() for _ in chains]
    errors, equal = [], []
    start = threading.Barrier(2)
    torch.cuda.synchronize()

    def worker(i):
        try:
            ctxs[i].bind()
            with torch.cuda.stream(streams[i]):
                start.wait()
                for _ in range(6):
                    chains[i].reset()
                    chains[i].run(streams[i])
                    got = chains[i].state()
                    streams[i].synchronize()
                    equal.append(_same(got, want[i]))
                fs.check_device_status(streams[i])
        except Exception as e:  # reported in the main thread
            errors.append(e)
        finally:
            fs.Context.unbind()

    th = [threading.Thread(target=worker, args=(i,)) for i in range(2)]
    for x in th:
        x.start()
    for x in th:
        x.join()
    for c in ctxs:
        c.destroy()
    assert not errors, errors
    assert equal == [True] * 12


def test_two_graphs_share_the_workspace(fs):
    """Chains captured as two graphs of one context, replayed in turns on one
    stream, give what the eager calls give."""
    chains = _chains(fs)
    want = [c.eager() for c in chains]
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    graphs = []
    with torch.cuda.stream(s):
        for c in chains:
            fs.capture_begin(s)
            c.run(s)
            graphs.append(fs.capture_end(s))
        for turn in (0, 1, 1, 0, 1):
            chains[turn].reset()
            graphs[turn].replay(s)
            got = chains[turn].state()
            s.synchronize()
            assert _same(got, want[turn]), turn
    fs.check_device_status(s)
    for g in graphs:
        g.destroy()


def test_batch_cut_by_the_workspace(fs):
    """With weights, 16 heads x 400000 tokens leave room for two rows' scores:
    a batch of three runs as two rows and one, and equals those calls."""
    from rank_transformer_b200.kv8 import KV8Cache
    G, rep, D, S_max = 1, 16, 64, 400000
    n = [300, 70, 129]
    k, v = _normal(1, 3, 301, G, D), _normal(2, 3, 301, G, D)
    q, kn, vn = _normal(3, 3, rep, D), _normal(4, 3, G, D), _normal(5, 3, G, D)
    dn = torch.tensor(n, dtype=torch.int32, device="cuda")

    def run(rows):
        B = len(rows)
        c = KV8Cache(B, G, D, S_max)
        fs.kv8_store(k[rows].contiguous(), v[rows].contiguous(), c, dn[rows].contiguous(), 301, 301)
        w = torch.full((B, G, S_max), 2.0, device="cuda")
        out = torch.zeros((B, rep, D), dtype=torch.bfloat16, device="cuda")
        before = fs.lib.flashsvd_launch_count()
        fs.kv8_decode_attn(q[rows].contiguous(), kn[rows].contiguous(), vn[rows].contiguous(), c,
                           dn[rows].contiguous(), w, True, out, rep, 0.125)
        launches = fs.lib.flashsvd_launch_count() - before
        torch.cuda.synchronize()
        fs.check_device_status()
        return out, w, launches

    out, w, launches = run([0, 1, 2])
    assert launches == 4
    o2, w2, l2 = run([0, 1])
    o1, w1, l1 = run([2])
    assert (l2, l1) == (2, 2)
    assert torch.equal(out, torch.cat([o2, o1])) and torch.equal(w, torch.cat([w2, w1]))
    for b in range(3):
        assert (w[b, :, n[b] + 1:] == 2.0).all()
        # the probabilities of 16 heads; the appended token's are set, the others added to 2
        total = w[b, :, :n[b] + 1].double().sum() - 2.0 * n[b]
        assert abs(total - rep) < 1e-3  # 300 entries near 2, half a step of fp32 (2^-23) each, and 2^-20 a head


@pytest.mark.parametrize("fmt", ["int8", "e4m3"])
@pytest.mark.parametrize("D", [64, 128])
def test_evict_scales_far_apart(fs, fmt, D):
    """Blocks whose scale was set by a row that goes: the codes of the others
    move by every power of two, up to where none is left, next to codes of
    blocks whose scale hardly changes, and back down again."""
    from tests.test_kv8_gpu import _bf16, _cache, _check_cache, _dev, _host
    G, n, keep = 26, 256, 150
    rng = np.random.default_rng(11)
    x = [rng.standard_normal((1, n, G, D)) * 2.0 ** rng.integers(-3, 1, size=(1, n, G, D)) for _ in range(2)]
    for g in range(G):
        for blk, gap in enumerate((g, 7 * g % G, 25 - g)):
            for t in x:
                t[0, 64 * blk, g] = 2.0 ** gap * (1 + rng.random(D))
    k, v = (_bf16(t) for t in x)
    w = np.ones((1, G, 256), np.float32)
    w[:, :, [0, 64, 128]] = 0.0
    w[:, :, 153:] = 0.5
    idx = oracle.evict_kept(w[0, 0].astype(np.float64), keep, 0)
    assert not set(idx) & {0, 64, 128} and len(idx) == keep
    for in_place in (False, True):
        src = _cache(fs, 1, G, D, n, fmt)
        fs.kv8_store(_dev(k), _dev(v), src, None, n, n)
        dst = src if in_place else _cache(fs, 1, G, D, n, fmt, 0x11)
        before = _host(dst)
        wd = torch.from_numpy(w.copy()).cuda()
        nd = torch.tensor([n], dtype=torch.int32, device="cuda")
        kept = torch.zeros((1, G, keep), dtype=torch.int32, device="cuda")
        fs.kv8_evict(src, dst, wd, wd if in_place else torch.zeros_like(wd), nd, None, kept, keep, 0)
        torch.cuda.synchronize()
        fs.check_device_status()
        host = _host(dst)
        for g in range(G):
            for i, t in enumerate((k, v)):
                _check_cache(host, before, i, 0, g, oracle.kv8_rows(t[0, :, g], fmt)[idx], fmt)


@pytest.mark.parametrize("B,S,G,rep,D,window,lens", [
    (2, 2100, 2, 3, 64, 40, [2100, 130]),      # 7 parts a row tile; most of the short row's are empty
    (1, 1500, 1, 1, 128, 1500, None),          # parts in front of, on and behind the diagonal
    (3, 1025, 1, 2, 64, 97, [1, 0, 1025]),
    (1, 4500, 1, 1, 128, 1, [4437]),
])
def test_weight_sums_in_parts(fs, B, S, G, rep, D, window, lens):
    """Few rows of many keys: the statistics' keys are cut into parts."""
    from tests.test_kv8_gpu import _bf16, _dev, _sums_bound
    rng = np.random.default_rng(S)
    H, scale = G * rep, D ** -0.5
    q, k = _bf16(1.5 * rng.standard_normal((B, S, H, D))), _bf16(rng.standard_normal((B, S, G, D)))
    n = lens or [S] * B
    for b in range(B):
        q[b, n[b]:], k[b, n[b]:] = np.nan, np.inf
    w = torch.full((B, G, S), 7.0, device="cuda")
    dl = None if lens is None else torch.tensor(lens, dtype=torch.int32, device="cuda")
    fs.attn_weight_sums(_dev(q), _dev(k), w, dl, B, S, H, G, D, S, S, window, scale)
    torch.cuda.synchronize()
    fs.check_device_status()
    got = w.double().cpu().numpy()
    for b in range(B):
        assert (got[b, :, n[b]:] == 7.0).all()
        for g in range(G if n[b] else 0):
            qq, kk = q[b, :n[b], g * rep:(g + 1) * rep], k[b, :n[b], g]
            want = oracle.attn_weight_sums(qq, kk, window, scale)
            assert np.all(np.abs(got[b, g, :n[b]] - want) <= _sums_bound(qq, kk, scale, window, want, D)), (b, g)


def test_refusals(fs):
    """Nothing is launched: the counter of launches stays."""
    from rank_transformer_b200.kv8 import KV8Cache
    L, P = fs.lib, fs.ptr
    c, d = KV8Cache(2, 2, 64, 256), KV8Cache(2, 2, 64, 256)
    x = torch.zeros((2, 64, 34, 64), dtype=torch.bfloat16, device="cuda")
    w, wo = torch.zeros((2, 2, 256), device="cuda"), torch.zeros((2, 2, 256), device="cuda")
    n = torch.zeros(2, dtype=torch.int32, device="cuda")
    kept = torch.zeros((2, 2, 256), dtype=torch.int32, device="cuda")
    before = L.flashsvd_launch_count()

    def attend(cache=c, q=x, kn=x, vn=x, seq=n, weights=None, out=x, H=4, scale=0.125):
        return L.flashsvd_kv8_decode_attn(P(q), P(kn), P(vn), cache.struct, P(seq), P(weights), 1, P(out), H, scale,
                                          None)
    assert attend(H=3) == INVALID and attend(H=0) == INVALID
    assert attend(H=34) == UNSUPPORTED
    assert attend(seq=None) == INVALID and attend(kn=None) == INVALID and attend(vn=None) == INVALID
    assert attend(scale=0.0) == INVALID and attend(scale=float("nan")) == INVALID
    assert attend(q=x.view(-1)[4:]) == MISALIGNED and attend(out=None) == INVALID
    many = KV8Cache(1025, 1, 64, 64)
    assert attend(cache=many, H=1) == UNSUPPORTED
    wide = KV8Cache(1, 1, 64, 1048640)  # 16 heads' scores of one row pass 2^24 floats
    assert attend(cache=wide, H=16, weights=torch.zeros((1, 1, 1048640), device="cuda")) == UNSUPPORTED

    def sums(B=2, S=64, H=4, G=2, D=64, S_max=64, stride=256, window=8, scale=0.125, weights=w):
        return L.flashsvd_attn_weight_sums(P(x), P(x), P(weights), None, B, S, H, G, D, S_max, stride, window, scale,
                                           None)
    assert sums(H=3) == INVALID and sums(S_max=63) == INVALID and sums(stride=63) == INVALID
    assert sums(window=0) == INVALID and sums(scale=-1.0) == INVALID and sums(weights=None) == INVALID
    assert sums(D=96) == UNSUPPORTED

    def evict(src=c, dst=d, wi=w, wout=wo, keep=100, recent=0, k=kept):
        return L.flashsvd_kv8_evict(src.struct, dst.struct, P(wi), P(wout), P(n), None, P(k), keep, recent, None)
    assert evict(keep=0) == INVALID and evict(keep=257) == INVALID and evict(recent=101) == INVALID
    assert evict(recent=-1) == INVALID and evict(k=None) == INVALID
    assert evict(dst=KV8Cache(2, 2, 64, 64)) == INVALID
    assert evict(dst=KV8Cache(2, 2, 64, 256, "e4m3")) == INVALID
    assert evict(dst=KV8Cache(2, 1, 64, 256)) == INVALID
    assert evict(wout=w) == INVALID and evict(dst=c) == INVALID  # in place in part
    shared = KV8Cache.from_tensors(d.k, d.v, d.k_scale, d.v_scale, d.k_tail, c.v_tail)
    crossed = KV8Cache.from_tensors(c.v, c.k, d.k_scale, d.v_scale, d.k_tail, d.v_tail)
    assert evict(dst=shared) == INVALID and evict(dst=crossed) == INVALID
    both = torch.zeros(2 * 2 * 256 + 128, device="cuda")
    assert evict(wi=both[:1024].view(2, 2, 256), wout=both[128:].view(2, 2, 256)) == INVALID
    inside = KV8Cache.from_tensors(c.k[:, :, :128].contiguous(), d.v[:, :, :128].contiguous(),
                                   c.k.view(torch.float32).view(-1)[:8].view(2, 2, 2),
                                   d.v_scale[:, :, :2].contiguous(), d.k_tail, d.v_tail)
    assert evict(dst=inside) == INVALID  # dst's scales within src's codes
    assert L.flashsvd_launch_count() == before
