"""The 8-bit cache through the layer and model entry points: prefill, decode
steps, eviction and decoding on, as a serving loop runs them."""
import math

import numpy as np
import pytest

from oracle import flashsvd_oracle as oracle
from rank_transformer_b200 import synth
from tests.gpu_util import assert_parity, dev_bf16, host_f64
from tests.test_layers_gpu import _decoder_struct, _rope

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")


@pytest.fixture(scope="module")
def fs():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from rank_transformer_b200 import flashsvd
    flashsvd.init(0, max_tokens=1024, max_rank=512, max_hidden=1024, max_ffn=2048)
    return flashsvd


def _values(c, which, n):
    """The n cached rows of every head, [B, G, n, D] float64."""
    codes, scale, tail = {"k": (c.k, c.k_scale, c.k_tail), "v": (c.v, c.v_scale, c.v_tail)}[which]
    x = codes.float() * scale.repeat_interleave(64, dim=2)[..., None]
    first = (n - 1) // 64 * 64
    return torch.cat([x[:, :, :first], tail[:, :, :n - first].float()], 2).double().cpu().numpy()


@pytest.mark.parametrize("fmt", ["int8", "e4m3"])
@pytest.mark.parametrize("B,S,window", [(1, 128, 128), (2, 100, 33)])
def test_layer_prefill_then_decode(fs, fmt, B, S, window):
    """Prefill output and rows equal those of the bf16 layer bit for bit, the
    cache holds them quantised, the weights are the oracle's within bf16
    rounding of q and k; each decode step against the oracle over the cached
    values, with rotary positions that differ from the cache's."""
    from rank_transformer_b200.kv8 import KV8Cache
    d, H, D, f, r, steps, S_max = 256, 4, 64, 688, 64, 30, 192
    rng = synth.rng_for(4 + S)
    w = synth.decoder_layer_weights(rng, d, f, r, r, gain_jitter=0.1)
    rows = S + steps + 50
    cos_t, sin_t = _rope(fs, rows, D)
    L, dev = _decoder_struct(fs, w, d, H, D, f, cos_t, sin_t)
    wf = oracle.widen_layer(w)
    xs = synth.normal_bf16(rng, (B, S + steps, d))

    kc = torch.zeros((B, S, H, D), dtype=torch.bfloat16, device="cuda")
    vc = torch.zeros_like(kc)
    x = dev_bf16(xs[:, :S].reshape(B * S, d))
    fs.layer_forward(L, x, kc, vc, None, B, S, S, fs.PREFILL_CAUSAL)
    c = KV8Cache(B, H, D, S_max, fmt)
    x8 = dev_bf16(xs[:, :S].reshape(B * S, d))
    k8, v8 = torch.zeros_like(kc), torch.zeros_like(kc)
    weights = torch.full((B, H, S_max), -1.0, device="cuda")
    fs.layer_forward_kv8(L, x8, c, k8, v8, weights, window, None, None, rows, B, S, fs.PREFILL_CAUSAL)
    torch.cuda.synchronize()
    fs.check_device_status()
    assert torch.equal(x, x8) and torch.equal(kc, k8) and torch.equal(vc, v8)
    hk, hv = host_f64(kc), host_f64(vc)
    got_k, got_v, got_w = _values(c, "k", S), _values(c, "v", S), weights.double().cpu().numpy()
    assert (got_w[:, :, S:] == -1.0).all()
    for b in range(B):
        n1 = oracle.rmsnorm(oracle.from_bf16(xs[b, :S]), wf["g1"])
        q = oracle.lowrank_linear(n1, wf["U_q"], wf["V_q"]).reshape(S, H, D)
        q = np.transpose(oracle.rope(np.transpose(q, (1, 0, 2)), np.arange(S)), (1, 0, 2))
        for h in range(H):
            np.testing.assert_array_equal(got_k[b, h], oracle.kv8_rows(hk[b, :, h], fmt))
            np.testing.assert_array_equal(got_v[b, h], oracle.kv8_rows(hv[b, :, h], fmt))
            want = oracle.attn_weight_sums(q[:, h:h + 1], hk[b, :, h], window, 1 / math.sqrt(D))
            assert_parity(got_w[b, h, :S], want, f"weights b={b} h={h}")
            # every query hands out one
            assert abs(got_w[b, h, :S].sum() - min(window, S)) < 1e-4 * min(window, S)

    shift = 37                       # rotary position minus place in the cache
    seq = torch.full((B,), S, dtype=torch.int32, device="cuda")
    pos = seq + shift
    k1, v1 = (torch.zeros((B, H, D), dtype=torch.bfloat16, device="cuda") for _ in range(2))
    kd = torch.zeros((B, rows, H, D), dtype=torch.bfloat16, device="cuda")
    vd = torch.zeros_like(kd)
    before = weights.clone()
    for t in range(steps):
        n = S + t
        hist_k = np.transpose(_values(c, "k", n), (0, 2, 1, 3))
        hist_v = np.transpose(_values(c, "v", n), (0, 2, 1, 3))
        xt = dev_bf16(xs[:, n])
        fs.layer_forward_kv8(L, xt, c, k1, v1, weights, 0, seq, pos, rows, B, 1, fs.DECODE)
        # the same token's rows from the bf16 layer at that position
        xd = dev_bf16(xs[:, n])
        fs.set_decode_path(False)
        fs.layer_forward(L, xd, kd, vd, pos, B, 1, rows, fs.DECODE)
        fs.set_decode_path(True)
        torch.cuda.synchronize()
        assert torch.equal(k1, kd[:, n + shift]) and torch.equal(v1, vd[:, n + shift])
        for b in range(B):
            n1 = oracle.rmsnorm(oracle.from_bf16(xs[b, n])[None], wf["g1"])
            q = oracle.lowrank_linear(n1, wf["U_q"], wf["V_q"]).reshape(H, 1, D)
            q = np.transpose(oracle.rope(q, np.array([n + shift])), (1, 0, 2))
            k = np.concatenate([hist_k[b], host_f64(k1)[b][None]])
            v = np.concatenate([hist_v[b], host_f64(v1)[b][None]])
            att = np.stack([oracle.attention_probs(q[:, h], k[:, h], 1 / math.sqrt(D))[0] @ v[:, h] for h in range(H)])
            hmid = oracle.from_bf16(xs[b, n]) + oracle.lowrank_linear(att.reshape(1, d), wf["U_o"], wf["V_o"])[0]
            n2 = oracle.rmsnorm(hmid[None], wf["g2"])
            y = hmid + oracle.packed_gateup_mlp(n2, wf["U_gu"], wf["V_gu"], wf["U_dn"], wf["V_dn"], r)[0]
            assert_parity(host_f64(xt)[b], y, f"decode step {t} b={b}")
        fs.advance_seqlens(seq, B)
        fs.advance_seqlens(pos, B)
    torch.cuda.synchronize()
    fs.check_device_status()
    n = S + steps
    # each step handed out one more per head, to tokens of the cache only
    gain = weights[:, :, :n].double().sum(-1) - before[:, :, :S].double().sum(-1)
    assert torch.allclose(gain, torch.full_like(gain, steps), rtol=0, atol=1e-3)
    assert (weights[:, :, n:] == -1.0).all()


def _model(fs, fmt, **kw):
    from rank_transformer_b200.model import DecoderConfig, DecoderModel
    cfg = DecoderConfig(layers=2, d=256, H=4, D=64, f=704, vocab=1000, rho=(0.5,))
    return DecoderModel(cfg, B=2, S_max=192, seed=3, kv_format=fmt, **kw)


@pytest.mark.parametrize("fmt", ["int8", "e4m3"])
def test_model_steps_and_graph(fs, fmt):
    """generate() past the cache's size: graph replay and eager steps give the
    same tokens, logits, caches and weights bit for bit, through two
    evictions."""
    prompt = torch.randint(0, 1000, (2, 150), dtype=torch.int32, generator=torch.Generator().manual_seed(1))
    a, b = (_model(fs, fmt, kv_keep=100, kv_recent=20, max_positions=400) for _ in range(2))
    stream = torch.cuda.Stream()
    b.capture(stream)
    assert b.step_graph.kernels > 0
    torch.cuda.synchronize()
    with torch.cuda.stream(stream):
        tokens = b.generate(prompt, 170, stream)
    stream.synchronize()
    a.prefill(prompt.cuda())
    mine = []
    for _ in range(170):
        mine.append(a.tokens.clone())
        a._make_room()
        a.decode_step_eager()
    torch.cuda.synchronize()
    fs.check_device_status()
    assert torch.equal(torch.stack(mine, 1).cpu(), tokens)
    assert a.position == b.position == 320 and a.length == b.length == 150 + 170 - 2 * 92
    assert a.seqlens.tolist() == [a.length] * 2 and a.positions.tolist() == [320] * 2
    assert torch.equal(a.logits, b.logits)
    for i in range(2):
        for x, y in zip(a.kv8[i].tensors(), b.kv8[i].tensors()):
            assert torch.equal(x.view(torch.uint8), y.view(torch.uint8))
        assert torch.equal(a.kv_weights[i], b.kv_weights[i])
    b.release_graphs()


def test_model_eviction_keeps_the_oracle_s_tokens(fs):
    m = _model(fs, "int8", kv_keep=70, kv_recent=7)
    prompt = torch.randint(0, 1000, (2, 180), dtype=torch.int32, generator=torch.Generator().manual_seed(2))
    m.prefill(prompt.cuda())
    for _ in range(5):
        m.decode_step_eager()
    torch.cuda.synchronize()
    n = 185
    w = [x[:, :, :n].double().cpu().numpy() for x in m.kv_weights]
    rows = [(_values(c, "k", n), _values(c, "v", n)) for c in m.kv8]
    m.evict()
    torch.cuda.synchronize()
    fs.check_device_status()
    assert m.seqlens.tolist() == [70, 70] and m.length == 70 and m.position == 185
    for i, c in enumerate(m.kv8):
        for x, which in enumerate(("k", "v")):
            got = _values(c, which, 70)
            for b in range(2):
                for h in range(4):
                    idx = oracle.evict_kept(w[i][b, h], 70, 7)
                    np.testing.assert_array_equal(got[b, h], oracle.kv8_rows(rows[i][x][b, h][idx], "int8"))
    m.evict()                       # nothing left to drop
    assert m.seqlens.tolist() == [70, 70]
    m.decode_step_eager()
    torch.cuda.synchronize()
    assert torch.isfinite(m.logits).all()


def test_model_refusals(fs):
    with pytest.raises(ValueError):
        _model(fs, None, kv_keep=10)
    with pytest.raises(ValueError):
        _model(fs, "int8", kv_keep=192)
    with pytest.raises(ValueError):
        _model(fs, "int8", kv_keep=100, kv_recent=101)
    with pytest.raises(ValueError):
        _model(fs, "int8", max_positions=100)
    with pytest.raises(ValueError):
        _model(fs, "int4")
    m = _model(fs, "int8")
    with pytest.raises(ValueError):
        m.evict()
    m.prefill(torch.zeros((2, 190), dtype=torch.int32, device="cuda"))
    m.capture(torch.cuda.Stream())
    with pytest.raises(ValueError):      # 190 + 3 tokens do not fit 192
        m.generate(torch.zeros((2, 190), dtype=torch.int32), 3)
    torch.cuda.synchronize()
    m.release_graphs()


def test_layer_refusals(fs):
    from rank_transformer_b200.kv8 import KV8Cache
    d, H, D, f, r = 256, 4, 64, 688, 64
    w = synth.decoder_layer_weights(synth.rng_for(1), d, f, r, r)
    cos_t, sin_t = _rope(fs, 200, D)
    L, dev = _decoder_struct(fs, w, d, H, D, f, cos_t, sin_t)
    c = KV8Cache(2, H, D, 128, "int8")
    x = torch.zeros((2 * 128, d), dtype=torch.bfloat16, device="cuda")
    rows = torch.zeros_like(x)
    seq = torch.zeros(2, dtype=torch.int32, device="cuda")
    weights = torch.zeros((2, H, 128), device="cuda")

    def status(**kw):
        a = dict(cache=c, weights=weights, window=5, seq=seq, pos=None, rope_rows=200, B=2, S=128,
                 mode=fs.PREFILL_CAUSAL)
        a.update(kw)
        try:
            fs.layer_forward_kv8(L, x, a["cache"], rows, rows, a["weights"], a["window"], a["seq"], a["pos"],
                                 a["rope_rows"], a["B"], a["S"], a["mode"])
        except fs.FlashSVDError as e:
            return e.status
        return 0

    assert status(S=0) == 0
    assert status(B=1) == 1                                   # the cache's batch is 2
    assert status(S=129) == 1 and status(rope_rows=127) == 1 and status(rope_rows=0) == 1
    assert status(window=0) == 1 and status(mode=fs.ENCODER_BIDIR) == 1
    assert status(cache=KV8Cache(2, 2, D, 128, "int8")) == 1
    assert status(cache=KV8Cache(2, H, 128, 128, "int8")) == 1
    assert status(mode=fs.DECODE, S=2) == 1 and status(mode=fs.DECODE, S=1, seq=None) == 1
    torch.cuda.synchronize()
