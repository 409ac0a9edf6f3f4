"""GPU parity of the 8-bit key/value cache (store, decode attention with
weight accumulation, prompt weight sums, eviction) against the float64
oracle, called through the C ABI.

What is compared exactly: codes, scales, tails, kept indices, moved weights
(the definitions leave no rounding open).  Attention outputs and weights have
bounds derived in `_attend_bound` and `_sums_bound`.
"""
import math

import numpy as np
import pytest

from oracle import flashsvd_oracle as oracle

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")

U32 = 2.0 ** -24      # half a step of fp32


@pytest.fixture(scope="module")
def fs():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from rank_transformer_b200 import flashsvd
    flashsvd.init(0, max_tokens=512, max_rank=512, max_hidden=1024, max_ffn=2048)
    return flashsvd


def _bf16(a):
    """Round to bf16 numbers, as float64."""
    return torch.from_numpy(np.asarray(a, np.float32)).to(torch.bfloat16).double().numpy()


def _dev(a, dtype=torch.bfloat16):
    return torch.from_numpy(np.array(a)).to(dtype).cuda()


def _rows(rng, shape, spread=True):
    """Random rows; with `spread`, blocks of very different magnitude."""
    x = rng.standard_normal(shape)
    if spread:
        x = x * 2.0 ** rng.integers(-6, 7, size=shape[:-1] + (1,))
    return _bf16(x)


def _cache(fs, B, G, D, S_max, fmt, fill=0x5a):
    """A cache whose every byte is set, so that what a call must leave alone
    can be told."""
    from rank_transformer_b200.kv8 import KV8Cache
    c = KV8Cache(B, G, D, S_max, fmt)
    for t in c.tensors():
        t.view(torch.uint8).fill_(fill)
    return c


def _host(c):
    k, v, ks, vs, kt, vt = c.tensors()
    return [dict(codes=a.float().cpu().double().numpy(), scale=s.cpu().double().numpy(),
                 tail=t.cpu().double().numpy()) for a, s, t in ((k, ks, kt), (v, vs, vt))]


def _check_cache(host, before, x, b, g, rows, fmt):
    """Tensor x (0 keys, 1 values) of one head holds `rows` [n, D] and nothing
    else has changed."""
    n = rows.shape[0]
    h, old = host[x], before[x]
    full = n // 64
    for blk in range(full):
        codes, s = oracle.kv8_block(rows[64 * blk:64 * blk + 64], fmt)
        np.testing.assert_array_equal(h["codes"][b, g, 64 * blk:64 * blk + 64], codes)
        np.testing.assert_array_equal(h["scale"][b, g, blk], s)
    np.testing.assert_array_equal(h["codes"][b, g, 64 * full:], old["codes"][b, g, 64 * full:])
    np.testing.assert_array_equal(h["scale"][b, g, full:], old["scale"][b, g, full:])
    first = (n - 1) // 64 * 64 if n else 0
    np.testing.assert_array_equal(h["tail"][b, g, :n - first], rows[first:])
    np.testing.assert_array_equal(h["tail"][b, g, n - first:], old["tail"][b, g, n - first:])


# ------------------------------------------------------------------- store --

@pytest.mark.parametrize("fmt", ["int8", "e4m3"])
@pytest.mark.parametrize("B,G,D,S,S_src,S_max,lens", [
    (1, 1, 64, 1, 1, 64, None),
    (1, 3, 128, 63, 70, 64, None),
    (2, 2, 64, 64, 64, 128, None),
    (2, 1, 128, 129, 129, 192, [129, 65]),
    (4, 5, 64, 200, 201, 256, [0, 64, 200, 1]),
    (3, 2, 128, 130, 130, 192, [-5, 128, 999]),
])
def test_store(fs, fmt, B, G, D, S, S_src, S_max, lens):
    rng = np.random.default_rng(10 * S + D)
    k, v = _rows(rng, (B, S_src, G, D)), _rows(rng, (B, S_src, G, D))
    n = [S] * B if lens is None else [min(max(x, 0), S) for x in lens]
    for b in range(B):   # rows behind a sequence hold anything
        k[b, n[b]:], v[b, n[b]:] = math.nan, math.inf
    c = _cache(fs, B, G, D, S_max, fmt)
    before = _host(c)
    dl = None if lens is None else _dev(lens, torch.int32)
    fs.kv8_store(_dev(k), _dev(v), c, dl, S, S_src)
    torch.cuda.synchronize()
    host = _host(c)
    for b in range(B):
        for g in range(G):
            for x, rows in ((0, k), (1, v)):
                _check_cache(host, before, x, b, g, rows[b, :n[b], g], fmt)


@pytest.mark.parametrize("fmt", ["int8", "e4m3"])
def test_store_edge_values(fs, fmt):
    """Zero, subnormal, huge, just-fitting and non-finite blocks."""
    D, lim = 64, oracle.KV8_LIMIT[fmt]
    rng = np.random.default_rng(1)
    x = _bf16(rng.standard_normal((1, 64 * 8, 1, D)))
    x[0, 0:64] = 0.0
    x[0, 64:128] *= 2.0 ** -110
    x[0, 128:192] *= 2.0 ** 120
    x[0, 192:256] = np.clip(x[0, 192:256], -0.9, 0.9)
    x[0, 192, 0, 0] = lim / 128                     # fits exactly
    x[0, 256:320] = np.clip(x[0, 256:320], -0.9, 0.9)
    x[0, 256, 0, 0] = -255.0 / 64                   # one code too many for 127
    x[0, 320, 0, 3] = math.nan
    x[0, 384, 0, 3] = -math.inf
    x[0, 448:] = np.where(rng.random((64, 1, D)) < 0.5, 63.5, 0.5)[:, :, :]  # ties
    x[0, 448, 0, 0] = 127.0
    x = np.where(np.isfinite(x), _bf16(np.where(np.isfinite(x), x, 0)), x)
    c = _cache(fs, 1, 1, D, 64 * 8, fmt)
    before = _host(c)
    fs.kv8_store(_dev(x), _dev(x), c, None, 512, 512)
    torch.cuda.synchronize()
    host = _host(c)
    _check_cache(host, before, 0, 0, 0, x[0, :, 0], fmt)
    _check_cache(host, before, 1, 0, 0, x[0, :, 0], fmt)


# --------------------------------------------------------------- attention --

def _attend_bound(q, kx, vx, p, scale, out):
    """Bounds on |out - exact| [D] and on |p - exact| / p for one head.
    Scores: D products summed in fp32 in any order, each step off by at most
    one unit (2^-23), times the scale factors (a few roundings): relative to
    sum |q k|.  A score off by d (natural units) moves p by a factor e^d, and
    the normalising sum by as much.  2^x and the sums add 2^-22 + n-independent
    fp32 steps (n additions of positive terms, split over >= 8 lanes).  The
    probabilities are rounded to 11 bits (2^-11 each, and below 2^-40 of the
    largest dropped), the output to bf16 (2^-8)."""
    n, D = kx.shape
    d = scale * (np.abs(kx) @ np.abs(q)) * (D + 16) * 2 * U32 + np.abs(kx @ q) * scale * 8 * U32
    eps_p = 2 * d.max() + (n / 8 + 64) * 2 * U32 + 2.0 ** -20
    av = np.abs(vx)
    e_out = (eps_p + 2.0 ** -11) * (p @ av) + n * 2.0 ** -40 * av.max(0) + 2.0 ** -8 * np.abs(out)
    return e_out, eps_p


def _attend_case(fs, fmt, B, G, rep, D, S_max, pos, append, weights, accumulate, seed, check=True, qstd=1.5):
    rng = np.random.default_rng(seed)
    H = G * rep
    scale = 1.0 / math.sqrt(D)
    n = [min(max(x, 0), S_max - 1) for x in pos]     # tokens before the new one
    k = _rows(rng, (B, S_max, G, D), spread=False)
    v = _rows(rng, (B, S_max, G, D))
    q = _bf16(qstd * rng.standard_normal((B, H, D)))
    c = _cache(fs, B, G, D, S_max, fmt)
    held = [x if append else x + 1 for x in n]
    dk, dv = _dev(k), _dev(v)
    fs.kv8_store(dk, dv, c, _dev(held, torch.int32), S_max, S_max)
    torch.cuda.synchronize()
    before = _host(c)
    kn = np.stack([k[b, n[b]] for b in range(B)])
    vn = np.stack([v[b, n[b]] for b in range(B)])
    w0 = rng.random((B, G, S_max)).astype(np.float32)
    w = torch.from_numpy(w0.copy()).cuda() if weights else None
    out = torch.full((B, H, D), 7.0, dtype=torch.bfloat16, device="cuda")
    fs.kv8_decode_attn(_dev(q), _dev(kn) if append else None, _dev(vn) if append else None, c,
                       _dev(pos, torch.int32), w, accumulate, out, H, scale)
    torch.cuda.synchronize()
    fs.check_device_status()
    if not check:
        return out, w, c
    got, host = out.double().cpu().numpy(), _host(c)
    for b in range(B):
        for g in range(G):
            kr, vr = k[b, :n[b] + 1, g], v[b, :n[b] + 1, g]
            if append:
                _check_cache(host, before, 0, b, g, kr, fmt)
                _check_cache(host, before, 1, b, g, vr, fmt)
            kx, vx = oracle.kv8_rows(kr, fmt), oracle.kv8_rows(vr, fmt)
            add = np.zeros(n[b] + 1)
            worst = 0.0
            for h in range(g * rep, (g + 1) * rep):
                p = oracle.attention_probs(q[b, h][None], kx, scale)[0]
                want = p @ vx
                e_out, eps_p = _attend_bound(q[b, h], kx, vx, p, scale, want)
                err = np.abs(got[b, h] - want)
                assert np.all(err <= e_out), (b, h, float(np.max(err / e_out)))
                add += p
                worst = max(worst, eps_p)
            if weights:
                wg = w[b, g].double().cpu().numpy()
                base = w0[b, g, :n[b] + 1].astype(np.float64) if accumulate else np.zeros(n[b] + 1)
                if append:
                    base[n[b]] = 0.0
                assert np.all(np.abs(wg[:n[b] + 1] - base - add) <= worst * add + 4 * U32 * (base + add) + 2.0 ** -100)
                np.testing.assert_array_equal(wg[n[b] + 1:], w0[b, g, n[b] + 1:])
    return out, w, c


ATTEND = [
    # B, G, rep, D, S_max, positions
    (1, 1, 1, 64, 64, [0]),
    (1, 1, 1, 128, 64, [63]),
    (1, 2, 1, 128, 128, [64]),
    (2, 1, 2, 64, 192, [127, 5]),
    (3, 2, 4, 128, 448, [0, 300, 447]),
    (2, 3, 7, 128, 640, [639, 320]),
    (2, 1, 8, 64, 1024, [1000, 575]),
    (1, 2, 9, 128, 320, [257]),
    (2, 2, 16, 64, 320, [191, 256]),
    (1, 1, 16, 128, 2048, [2047]),
    (40, 1, 1, 64, 128, [(37 * i) % 128 for i in range(40)]),
    (2, 32, 1, 128, 256, [200, 13]),
    (2, 2, 2, 64, 128, [-3, 5000]),
]


@pytest.mark.parametrize("fmt", ["int8", "e4m3"])
@pytest.mark.parametrize("case", range(len(ATTEND)))
def test_attend(fs, fmt, case):
    B, G, rep, D, S_max, pos = ATTEND[case]
    _attend_case(fs, fmt, B, G, rep, D, S_max, pos, True, case % 2 == 0, case % 4 == 0, 100 + case)
    _attend_case(fs, fmt, B, G, rep, D, S_max, pos, case % 2 == 1, True, case % 4 != 0, 200 + case)


@pytest.mark.parametrize("fmt", ["int8", "e4m3"])
def test_attend_sharp_and_far_maxima(fs, fmt):
    """Scores far apart (one key takes almost everything) and a large n."""
    _attend_case(fs, fmt, 1, 2, 4, 128, 4096, [4090], True, True, True, 7, qstd=20.0)
    _attend_case(fs, fmt, 2, 1, 12, 64, 4096, [4095, 17], True, True, False, 8, qstd=0.01)


def test_attend_equals_itself(fs):
    """The same call again gives the same bits, on another stream too."""
    o1, w1, _ = _attend_case(fs, "int8", 3, 4, 3, 128, 1024, [900, 64, 1023], True, True, False, 5, check=False)
    s = torch.cuda.Stream()
    with torch.cuda.stream(s):
        o2, w2, _ = _attend_case(fs, "int8", 3, 4, 3, 128, 1024, [900, 64, 1023], True, True, False, 5, check=False)
    torch.cuda.synchronize()
    assert torch.equal(o1, o2)
    for b, n in enumerate((901, 65, 1024)):
        assert torch.equal(w1[b, :, :n], w2[b, :, :n])


@pytest.mark.parametrize("fmt", ["int8", "e4m3"])
def test_steps_equal_store(fs, fmt):
    """A cache filled row by row holds what a stored prompt holds, bit for bit,
    and captured steps replay to the same."""
    B, G, D, n = 2, 2, 64, 150
    rng = np.random.default_rng(4)
    k, v = _dev(_rows(rng, (B, n, G, D))), _dev(_rows(rng, (B, n, G, D)))
    q = _dev(_bf16(rng.standard_normal((B, G * 2, D))))
    a, b_, c = (_cache(fs, B, G, D, 192, fmt, 0) for _ in range(3))
    fs.kv8_store(k, v, a, None, n, n)
    seq = torch.zeros(B, dtype=torch.int32, device="cuda")
    out = torch.empty((B, G * 2, D), dtype=torch.bfloat16, device="cuda")
    w = torch.zeros((B, G, 192), device="cuda")
    for t in range(n):
        fs.kv8_decode_attn(q, k[:, t].contiguous(), v[:, t].contiguous(), b_, seq, w, True, out, G * 2, 0.125)
        fs.advance_seqlens(seq, B)
    torch.cuda.synchronize()
    ha, hb = _host(a), _host(b_)
    for x in range(2):
        np.testing.assert_array_equal(ha[x]["codes"], hb[x]["codes"])
        np.testing.assert_array_equal(ha[x]["scale"], hb[x]["scale"])
        np.testing.assert_array_equal(ha[x]["tail"][:, :, :n - 128], hb[x]["tail"][:, :, :n - 128])
    # captured
    w2, out2 = torch.zeros_like(w), torch.empty_like(out)
    kn, vn = torch.empty_like(k[:, 0]), torch.empty_like(v[:, 0])
    seq.zero_()
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        fs.capture_begin(s)
        fs.kv8_decode_attn(q, kn, vn, c, seq, w2, True, out2, G * 2, 0.125, s)
        fs.advance_seqlens(seq, B, s)
        graph = fs.capture_end(s)
        assert graph.kernels == 3
        for t in range(n):
            kn.copy_(k[:, t])
            vn.copy_(v[:, t])
            graph.replay(s)
    s.synchronize()
    graph.destroy()
    assert torch.equal(out, out2) and torch.equal(w, w2)
    for x, y in zip(b_.tensors(), c.tensors()):
        assert torch.equal(x.view(torch.int8) if x.element_size() == 1 else x,
                           y.view(torch.int8) if y.element_size() == 1 else y)


@pytest.mark.parametrize("fmt", ["int8", "e4m3"])
def test_attend_non_finite(fs, fmt):
    """A NaN or an infinity in a cached row makes the outputs of its KV head
    NaN, and of no other; rows behind the sequence and unused tail slots may
    hold NaN."""
    B, G, D, n = 1, 3, 64, 200
    rng = np.random.default_rng(9)
    k, v = _rows(rng, (B, n, G, D), False), _rows(rng, (B, n, G, D), False)
    k[0, 70, 1, 5] = math.nan
    v[0, 10, 2, 5] = math.inf
    c = _cache(fs, B, G, D, 256, fmt, 0xff)    # 0xff bytes: NaN as bf16, fp32 and e4m3
    fs.kv8_store(_dev(k), _dev(v), c, None, n, n)
    q = _dev(_bf16(rng.standard_normal((B, G * 2, D))))
    out = torch.zeros((B, G * 2, D), dtype=torch.bfloat16, device="cuda")
    fs.kv8_decode_attn(q, None, None, c, _dev([n - 1], torch.int32), None, False, out, G * 2, 0.125)
    torch.cuda.synchronize()
    o = out.float()
    assert torch.isfinite(o[0, :2]).all() and torch.isnan(o[0, 2:4]).all() and torch.isnan(o[0, 4:]).all()


# -------------------------------------------------------------------- sums --

def _sums_bound(q, k, scale, window, want, D):
    """|weights - exact|: every p of the sum is off by the factor of
    `_attend_bound`'s scores and sums (both its own score and its row's
    log-sum), the sum itself by fp32 additions."""
    n = k.shape[0]
    m = max(np.abs(q[i, h]) @ np.abs(k).max(0) for i in range(max(0, n - window), n) for h in range(q.shape[1]))
    d = scale * m * (D + 24) * 2 * U32
    return want * (2 * d + 2.0 ** -19 + (n / 4 + 64) * 2 * U32) + 1e-30


SUMS = [
    # B, S, S_max, G, rep, D, window, lens
    (1, 1, 1, 1, 1, 64, 1, None),
    (1, 5, 9, 2, 1, 128, 100, None),
    (2, 64, 64, 1, 1, 128, 64, [64, 0]),
    (1, 65, 65, 1, 2, 64, 65, None),
    (2, 129, 140, 2, 1, 128, 1, [129, 128]),
    (3, 300, 300, 1, 3, 64, 70, [300, 299, 1]),
    (1, 257, 257, 4, 1, 128, 257, None),
    (2, 200, 256, 2, 5, 128, 128, [77, 200]),
    (1, 700, 700, 1, 1, 64, 33, None),
    (1, 640, 640, 1, 2, 128, 640, [-4]),
]


@pytest.mark.parametrize("case", range(len(SUMS)))
def test_weight_sums(fs, case):
    B, S, S_max, G, rep, D, window, lens = SUMS[case]
    rng = np.random.default_rng(300 + case)
    H, stride = G * rep, S + 3
    scale = 1.0 / math.sqrt(D)
    q, k = _bf16(1.5 * rng.standard_normal((B, S, H, D))), _rows(rng, (B, S_max, G, D), False)
    n = [S] * B if lens is None else [min(max(x, 0), S) for x in lens]
    for b in range(B):
        q[b, n[b]:], k[b, n[b]:] = math.nan, math.inf
    w0 = rng.random((B, G, stride)).astype(np.float32)
    w = torch.from_numpy(w0.copy()).cuda()
    for _ in range(2):
        fs.attn_weight_sums(_dev(q), _dev(k), w, None if lens is None else _dev(lens, torch.int32), B, S, H, G, D,
                            S_max, stride, window, scale)
    torch.cuda.synchronize()
    fs.check_device_status()
    got = w.double().cpu().numpy()
    for b in range(B):
        for g in range(G):
            np.testing.assert_array_equal(got[b, g, n[b]:], w0[b, g, n[b]:])
            if n[b] == 0:
                continue
            qq, kk = q[b, :n[b], g * rep:(g + 1) * rep], k[b, :n[b], g]
            want = oracle.attn_weight_sums(qq, kk, window, scale)
            err = np.abs(got[b, g, :n[b]] - want)
            bound = _sums_bound(qq, kk, scale, window, want, D)
            assert np.all(err <= bound), (b, g, float(np.max(err / bound)))


# ------------------------------------------------------------------- evict --

EVICT = [
    # B, G, D, S_max, tokens, keep, recent, dst S_max
    (1, 1, 64, 64, [2], 1, 0, 64),
    (1, 1, 128, 64, [64], 64, 0, 64),
    (2, 2, 64, 256, [200, 256], 100, 30, 128),
    (2, 1, 128, 256, [256, 100], 128, 0, 128),
    (3, 2, 64, 320, [300, 0, 129], 128, 128, 192),
    (2, 3, 128, 576, [576, 70], 321, 320, 576),
    (1, 2, 64, 2048, [2000], 1990, 5, 2048),
    (1, 1, 64, 4096, [4095], 64, 1, 64),
    (2, 1, 64, 128, [999, -1], 65, 3, 128),
    (2, 1, 64, 12032, [12000, 9001], 300, 10, 320),
    (1, 2, 64, 70016, [70001], 1000, 0, 1024),
]


@pytest.mark.parametrize("fmt", ["int8", "e4m3"])
@pytest.mark.parametrize("kind", ["random", "ties", "odd"])
@pytest.mark.parametrize("case", range(len(EVICT)))
def test_evict(fs, fmt, kind, case):
    B, G, D, S_max, tokens, keep, recent, S_dst = EVICT[case]
    if S_max > 10000 and fmt == "e4m3":
        pytest.skip("the selection does not see the format")
    rng = np.random.default_rng(500 + case)
    n = [min(max(x, 0), S_max) for x in tokens]
    k, v = _rows(rng, (B, S_max, G, D)), _rows(rng, (B, S_max, G, D))
    w = rng.random((B, G, S_max)).astype(np.float32)
    if kind == "ties":
        w = np.floor(w * 4).astype(np.float32) / 4 - 0.5
        w[w == 0] = np.where(rng.random((w == 0).sum()) < 0.5, 0.0, -0.0)
    if kind == "odd":
        r = rng.random(w.shape)
        w[r < 0.2], w[r > 0.9], w[(r > 0.8) & (r < 0.85)] = math.nan, math.inf, -math.inf
    src = _cache(fs, B, G, D, S_max, fmt)
    dk, dv = _dev(k), _dev(v)
    fs.kv8_store(dk, dv, src, _dev(n, torch.int32), S_max, S_max)
    want = {}
    for b in range(B):
        for g in range(G):
            idx = oracle.evict_kept(w[b, g, :n[b]].astype(np.float64), keep, recent)
            want[b, g] = (idx, oracle.kv8_rows(k[b, :n[b], g], fmt)[idx], oracle.kv8_rows(v[b, :n[b], g], fmt)[idx],
                          w[b, g, idx])
    for in_place in (False, True):
        dst = src if in_place else _cache(fs, B, G, D, S_dst, fmt, 0x33)
        before = _host(dst)
        wd = torch.from_numpy(w.copy()).cuda()
        wo = wd if in_place else torch.full((B, G, S_dst), 5.0, device="cuda")
        w_before = wo.cpu().numpy().copy()
        nd = _dev(tokens, torch.int32)
        no = nd if in_place else torch.full((B,), -7, dtype=torch.int32, device="cuda")
        kept = torch.full((B, G, keep), -9, dtype=torch.int32, device="cuda")
        fs.kv8_evict(src, dst, wd, wo, nd, no, kept, keep, recent)
        torch.cuda.synchronize()
        fs.check_device_status()
        host, kept, wo = _host(dst), kept.cpu().numpy(), wo.cpu().numpy()
        assert no.cpu().tolist() == [min(keep, x) for x in n]
        for b in range(B):
            for g in range(G):
                idx, kr, vr, wr = want[b, g]
                m = len(idx)
                assert kept[b, g, :m].tolist() == idx.tolist()
                assert (kept[b, g, m:] == -1).all()
                np.testing.assert_array_equal(wo[b, g, :m], wr)
                np.testing.assert_array_equal(wo[b, g, m:], w_before[b, g, m:])
                if in_place and n[b] <= keep:      # left as it was: full blocks keep their codes
                    for x in range(2):
                        for f in ("codes", "scale", "tail"):
                            np.testing.assert_array_equal(host[x][f][b, g], before[x][f][b, g])
                else:
                    _check_cache(host, before, 0, b, g, kr, fmt)
                    _check_cache(host, before, 1, b, g, vr, fmt)


def test_evict_selection_of_very_long_rows(fs):
    """Rows whose stretches do not fit in shared memory, with ties across
    them, against a stable sort."""
    S_max, keep, recent = 262144, 5000, 77
    g = torch.Generator(device="cuda")
    g.manual_seed(3)
    w = torch.floor(torch.rand((2, 1, S_max), generator=g, device="cuda") * 300)
    src, dst = (_cache(fs, 2, 1, 64, s, "int8", 0) for s in (S_max, 5056))
    n = torch.tensor([S_max, S_max - 12345], dtype=torch.int32, device="cuda")
    kept = torch.empty((2, 1, keep), dtype=torch.int32, device="cuda")
    wo = torch.zeros((2, 1, 5056), device="cuda")
    fs.kv8_evict(src, dst, w, wo, n, None, kept, keep, recent)
    torch.cuda.synchronize()
    fs.check_device_status()
    for b in range(2):
        m = int(n[b])
        first = torch.sort(w[b, 0, :m - recent], dim=0, descending=True, stable=True).indices[:keep - recent]
        want = torch.cat([torch.sort(first).values, torch.arange(m - recent, m, device="cuda")])
        assert torch.equal(kept[b, 0].long(), want)
        assert torch.equal(wo[b, 0, :keep], w[b, 0, want])


def test_evict_many_blocks_in_place(fs):
    """More blocks than can run at once, so that writers wait for readers;
    repeated, each time on a fresh copy."""
    B, G, D, S_max, keep, recent = 4, 8, 128, 8192, 6000, 100
    rng = np.random.default_rng(77)
    src = _cache(fs, B, G, D, S_max, "int8")
    k = torch.randn((B, S_max, G, D), device="cuda").to(torch.bfloat16)
    n = torch.full((B,), S_max - 7, dtype=torch.int32, device="cuda")
    w = torch.from_numpy(rng.random((B, G, S_max)).astype(np.float32)).cuda()
    kept, no = (torch.empty(s, dtype=torch.int32, device="cuda") for s in ((B, G, keep), (B,)))
    dst = _cache(fs, B, G, D, 6016, "int8", 0)
    wo = torch.zeros((B, G, 6016), device="cuda")
    for rep in range(3):
        fs.kv8_store(k, -k, src, n, S_max, S_max)
        fs.kv8_evict(src, dst, w, wo, n, no, kept, keep, recent)
        w2, n2, kept2 = w.clone(), n.clone(), torch.empty_like(kept)
        fs.kv8_evict(src, src, w2, w2, n2, n2, kept2, keep, recent)
        torch.cuda.synchronize()
        fs.check_device_status()
        assert torch.equal(kept, kept2) and torch.equal(no, n2) and torch.equal(w2[:, :, :keep], wo[:, :, :keep])
        full = keep // 64
        assert torch.equal(src.k[:, :, :full * 64], dst.k[:, :, :full * 64])
        assert torch.equal(src.v[:, :, :full * 64], dst.v[:, :, :full * 64])
        assert torch.equal(src.k_scale[:, :, :full], dst.k_scale[:, :, :full])
        assert torch.equal(src.v_scale[:, :, :full], dst.v_scale[:, :, :full])
        assert torch.equal(src.k_tail[:, :, :keep % 64], dst.k_tail[:, :, :keep % 64])
        assert torch.equal(src.v_tail[:, :, :keep % 64], dst.v_tail[:, :, :keep % 64])
