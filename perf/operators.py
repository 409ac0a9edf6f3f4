"""The 8-bit key/value cache operators, case by case: what is measured, on
which inputs, and each operator's plain form.

Four operators share one cache per layer.  Tokens are grouped into blocks of
64; a block of one head is held as 8-bit codes with one power-of-two scale,
and the rows of the newest token's block also stay in a bf16 tail:

  store    a prompt's key and value rows into the cache
  attend   one decode step: append the new rows, attend, add up the weights
  sums     the attention weight each prompt token got from the last queries
  evict    keep the tokens with the largest weights and the newest ones

``run`` computes the plain form with elementary torch operations, or, where
``own`` is true, calls the framework.
"""
import math

import torch

own = False

BLOCK = 64
LIMIT = {"int8": 127.0, "e4m3": 448.0}
DTYPE = {"int8": torch.int8, "e4m3": torch.float8_e4m3fn}


# ------------------------------------------------------------------- cases --

def listed():
    return [
        # a short prompt of a small model enters the cache: launch latency
        dict(name="store_s77_small", op="store", fmt="int8", B=1, G=4, D=64, S=77, ragged=False),
        # a 2048-token prompt of a 7B-shaped layer (32 heads of 128)
        dict(name="store_s2048_7b", op="store", fmt="int8", B=1, G=32, D=128, S=2048, ragged=False),
        # a padded batch of 16 prompts of unequal lengths, shared heads
        dict(name="store_ragged_b16", op="store", fmt="e4m3", B=16, G=8, D=128, S=4001, ragged=True),
        # one token of a small model over a short history: launch latency
        dict(name="attend_n100_small", op="attend", fmt="int8", B=1, G=4, H=4, D=64, N=100, ragged=False, weights=False),
        # one token of a 7B-shaped layer over 2048 cached tokens
        dict(name="attend_n2048_7b", op="attend", fmt="int8", B=1, G=32, H=32, D=128, N=2048, ragged=False, weights=False),
        # a serving batch of unequal histories up to 8192, four query heads a KV head
        dict(name="attend_b32_ragged", op="attend", fmt="e4m3", B=32, G=8, H=32, D=128, N=8191, ragged=True, weights=False),
        # four long histories, eight query heads a KV head, weights added up for eviction
        dict(name="attend_n131072", op="attend", fmt="int8", B=4, G=8, H=64, D=128, N=131071, ragged=False, weights=True),
        # all queries of a small model's prompt
        dict(name="sums_s300_small", op="sums", B=2, G=4, H=8, D=64, S=300, W=300, ragged=True),
        # all queries of a 2048-token prompt, 7B-shaped layer
        dict(name="sums_s2048_7b", op="sums", B=1, G=32, H=32, D=128, S=2048, W=2048, ragged=False),
        # an observation window at the end of long prompts, shared heads
        dict(name="sums_w64_s16000", op="sums", B=2, G=8, H=32, D=128, S=16000, W=64, ragged=False),
        # half of a 7B-shaped layer's 2048 tokens are dropped
        dict(name="evict_n2048_7b", op="evict", fmt="int8", B=1, G=32, D=128, N=2048, keep=1024, recent=256, ragged=False),
        # long histories brought down to a fixed budget
        dict(name="evict_n131072", op="evict", fmt="e4m3", B=4, G=8, D=128, N=131072, keep=32768, recent=1000, ragged=False),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["store", "attend", "attend", "sums", "evict"])
    fmt = rng.choice(["int8", "e4m3"])
    D = rng.choice([64, 128])
    G = rng.choice([1, 2, 4, 5, 8, 32])
    ragged = rng.random() < 0.5
    if op == "store":
        S = _log(rng, 1, 16000)
        B = max(1, min(rng.randint(1, 24), 290000 // (S * G)))
        return dict(op=op, fmt=fmt, B=B, G=G, D=D, S=S, ragged=ragged)
    if op == "attend":
        N = _log(rng, 1, 131071)
        rep = rng.choice([1, 2, 4, 7, 8, 16])
        B = max(1, min(rng.randint(1, 40), 4000000 // (N * G)))
        return dict(op=op, fmt=fmt, B=B, G=G, H=G * rep, D=D, N=N, ragged=ragged, weights=rng.random() < 0.5)
    if op == "sums":
        S = _log(rng, 1, 16000)
        W = _log(rng, 1, S) if rng.random() < 0.7 else S
        rep = rng.choice([1, 2, 4, 8])
        W = max(1, min(W, 65000000 // (S * G * rep)))
        B = max(1, min(rng.randint(1, 8), 65000000 // (S * W * G * rep)))
        return dict(op=op, B=B, G=G, H=G * rep, D=D, S=S, W=W, ragged=ragged)
    N = _log(rng, 2, 131072)
    B = max(1, min(rng.randint(1, 24), 4000000 // (N * G)))
    keep = rng.randint(1, max(1, min(N, 1000000 // (B * G))))
    recent = rng.randint(0, keep) if rng.random() < 0.8 else rng.choice([0, keep])
    return dict(op=op, fmt=fmt, B=B, G=G, D=D, N=N, keep=keep, recent=recent, ragged=ragged)


def _lens(case):
    """Tokens of each batch entry: N (or S), or unequal ones down to about a
    tenth of it."""
    n = case["N"] if "N" in case else case["S"]
    B = case["B"]
    return [max(1, n - (n * 9 * b) // (10 * B)) if case["ragged"] else n for b in range(B)]


def _up(n):
    return -(-n // BLOCK) * BLOCK


# --------------------------------------------------------- plain 8-bit form --

def _quantise(x, fmt):
    """Blocks x [..., 64, D] fp32 -> codes, scale [...]: the least power of
    two (at least 2^-100) with amax / scale <= the format's limit; a block
    with an infinity or NaN has the scale NaN and codes of zero."""
    amax = x.abs().amax((-2, -1))
    m, e = torch.frexp(amax)
    top, drop = (0.9921875, 7) if fmt == "int8" else (0.875, 9)
    k = torch.where(m <= top, e - drop, e - drop + 1)
    k = torch.where(amax > 0, k, torch.full_like(k, -100)).clamp(min=-100)
    ok = torch.isfinite(amax)
    k = torch.where(ok, k, torch.zeros_like(k))
    power = lambda t: ((t + 127) << 23).to(torch.int32).view(torch.float32)  # noqa: E731
    y = x * power(-k)[..., None, None]
    y = torch.where(ok[..., None, None], y, torch.zeros_like(y))
    codes = torch.round(y).to(torch.int8) if fmt == "int8" else y.to(torch.float8_e4m3fn)
    return codes, torch.where(ok, power(k), torch.full_like(amax, float("nan")))


def _values(codes, scale):
    """[B, G, S, D] codes and [B, G, S/64] scales -> fp32 values."""
    B, G, S, D = codes.shape
    x = codes.float().view(B, G, S // BLOCK, BLOCK, D) * scale[..., None, None]
    return x.view(B, G, S, D)


def _rows(c, which, n):
    """fp32 [B, G, S_max, D]: the rows of a cache that holds n[b] tokens; the
    newest token's block comes from the tail."""
    x = _values(c[which], c[which + "_scale"])
    B, G, S, D = x.shape
    blk = ((n - 1).clamp(min=0) // BLOCK)
    x = x.view(B, G, S // BLOCK, BLOCK, D)
    at = torch.arange(S // BLOCK, device=x.device)[None, None, :, None, None] == blk[:, None, None, None, None]
    return torch.where(at, c[which + "_tail"].float()[:, :, None], x).view(B, G, S, D)


def _set_rows(c, which, rows, n):
    """Write rows [B, G, S_max, D] fp32 (n[b] valid) into a cache: codes and
    scales of the full blocks, the newest token's block into the tail."""
    B, G, S, D = rows.shape
    nb = S // BLOCK
    blocks = rows.view(B, G, nb, BLOCK, D)
    full = (torch.arange(nb, device=rows.device)[None, :] + 1) * BLOCK <= n[:, None]
    full = full[:, None].expand(B, G, nb)
    fmt = c["fmt"]
    codes, scale = _quantise(torch.where(full[..., None, None], blocks, torch.zeros_like(blocks)), fmt)
    old = c[which].view(torch.int8).view(B, G, nb, BLOCK, D)
    old.copy_(torch.where(full[..., None, None], codes.view(torch.int8), old))
    c[which + "_scale"].copy_(torch.where(full, scale, c[which + "_scale"]))
    blk = (n - 1).clamp(min=0) // BLOCK
    last = torch.gather(blocks, 2, blk[:, None, None, None, None].expand(B, G, 1, BLOCK, D))[:, :, 0]
    slot = blk[:, None] * BLOCK + torch.arange(BLOCK, device=rows.device)[None, :] < n[:, None]
    tail = c[which + "_tail"]
    tail.copy_(torch.where(slot[:, None, :, None], last.to(torch.bfloat16), tail))


def _cache(B, G, D, S_max, fmt, device="cuda"):
    c = {"fmt": fmt}
    for w in ("k", "v"):
        c[w] = torch.zeros((B, G, S_max, D), dtype=torch.int8, device=device).view(DTYPE[fmt])
        c[w + "_scale"] = torch.zeros((B, G, S_max // BLOCK), dtype=torch.float32, device=device)
        c[w + "_tail"] = torch.zeros((B, G, BLOCK, D), dtype=torch.bfloat16, device=device)
    return c


def _state_of(c):
    return {w + s: c[w + s] for w in ("k", "v") for s in ("", "_scale", "_tail")}


# ------------------------------------------------------------------ inputs --

def _kv(shape, gen, which):
    """Rows as projections give them: unit normal, with a few strong channels
    in the keys."""
    x = torch.randn(shape, generator=gen, device="cuda", dtype=torch.float32)
    if which == "k":
        gain = torch.ones(shape[-1], device="cuda")
        gain[:: 16] = 3.0
        x *= gain
    return x


def _filled(case, n, gen):
    """A cache that holds n[b] tokens."""
    B, G, D = case["B"], case["G"], case["D"]
    c = _cache(B, G, D, _up(case["N"] + 1), case["fmt"])
    S = c["k"].shape[2]
    for w in ("k", "v"):
        _set_rows(c, w, _kv((B, G, S, D), gen, w).to(torch.bfloat16).float(), n)
    return c


def prepare(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    B, G, D, op = case["B"], case["G"], case["D"], case["op"]
    n = torch.tensor(_lens(case), dtype=torch.int32, device="cuda")
    s = {"case": case, "n": n}
    if op == "store":
        S = case["S"]
        for w in ("k", "v"):
            s[w] = _kv((B, S, G, D), gen, w).to(torch.bfloat16)
        s["cache"] = _cache(B, G, D, _up(S), case["fmt"])
    elif op == "attend":
        s["cache"] = _filled(case, n, gen)
        s["q"] = (1.5 * torch.randn((B, case["H"], D), generator=gen, device="cuda")).to(torch.bfloat16)
        s["k_new"] = _kv((B, G, D), gen, "k").to(torch.bfloat16)
        s["v_new"] = _kv((B, G, D), gen, "v").to(torch.bfloat16)
        s["weights"] = None
        if case["weights"]:
            S = s["cache"]["k"].shape[2]
            s["weights"] = torch.rand((B, G, S), generator=gen, device="cuda")
        s["out"] = torch.empty((B, case["H"], D), dtype=torch.bfloat16, device="cuda")
    elif op == "sums":
        S = case["S"]
        s["q"] = (1.5 * torch.randn((B, S, case["H"], D), generator=gen, device="cuda")).to(torch.bfloat16)
        s["k"] = _kv((B, S, G, D), gen, "k").to(torch.bfloat16)
        s["weights"] = torch.zeros((B, G, _up(S)), device="cuda")
    else:
        s["cache"] = _filled(case, n, gen)
        S = s["cache"]["k"].shape[2]
        # accumulated weights: heavy-tailed, some tokens never attended to
        w = torch.exp(2.0 * torch.randn((B, G, S), generator=gen, device="cuda"))
        s["weights"] = torch.where(torch.rand((B, G, S), generator=gen, device="cuda") < 0.05, torch.zeros_like(w), w)
        s["to"] = _cache(B, G, D, _up(case["keep"]), case["fmt"])
        s["weights_to"] = torch.zeros((B, G, _up(case["keep"])), device="cuda")
        s["n_to"] = torch.zeros(B, dtype=torch.int32, device="cuda")
        s["kept"] = torch.zeros((B, G, case["keep"]), dtype=torch.int32, device="cuda")
    if own:
        # what a user's program keeps: the library's workspace and the
        # handles of the caches (pointers and sizes of the tensors above)
        from rank_transformer_b200 import flashsvd as fs
        from rank_transformer_b200.kv8 import KV8Cache
        fs.init(0, max_tokens=64, max_rank=256, max_hidden=256, max_ffn=1024)
        for name in ("cache", "to"):
            if name in s:
                c = s[name]
                s[name + "_handle"] = KV8Cache.from_tensors(
                    c["k"], c["v"], c["k_scale"], c["v_scale"], c["k_tail"], c["v_tail"])
    return s


# --------------------------------------------------------------------- run --

def _scale_of(D):
    return 1.0 / math.sqrt(D)


def run(s):
    return (_run_own if own else _run_plain)(s)


def _run_own(s):
    from rank_transformer_b200 import flashsvd as fs
    case = s["case"]
    op = case["op"]
    if op == "store":
        fs.kv8_store(s["k"], s["v"], s["cache_handle"], s["n"], case["S"], case["S"])
        return _state_of(s["cache"])
    if op == "attend":
        fs.kv8_decode_attn(s["q"], s["k_new"], s["v_new"], s["cache_handle"], s["n"], s["weights"], True, s["out"],
                           case["H"], _scale_of(case["D"]))
        return {"out": s["out"], "weights": s["weights"], "cache": _state_of(s["cache"])}
    if op == "sums":
        fs.attn_weight_sums(s["q"], s["k"], s["weights"], s["n"], case["B"], case["S"], case["H"], case["G"],
                            case["D"], case["S"], s["weights"].shape[2], case["W"], _scale_of(case["D"]))
        return {"weights": s["weights"]}
    fs.kv8_evict(s["cache_handle"], s["to_handle"], s["weights"], s["weights_to"], s["n"], s["n_to"], s["kept"],
                 case["keep"], case["recent"])
    return {"kept": s["kept"], "n": s["n_to"], "weights": s["weights_to"], "cache": _state_of(s["to"])}


def _run_plain(s):
    return {"store": _plain_store, "attend": _plain_attend, "sums": _plain_sums, "evict": _plain_evict}[
        s["case"]["op"]](s)


def _plain_store(s):
    case, c = s["case"], s["cache"]
    S_max = c["k"].shape[2]
    pad = torch.zeros((case["B"], case["G"], S_max - case["S"], case["D"]), device="cuda")
    _set_rows(c, "k", torch.cat([s["k"].permute(0, 2, 1, 3).float(), pad], 2), s["n"])
    _set_rows(c, "v", torch.cat([s["v"].permute(0, 2, 1, 3).float(), pad], 2), s["n"])
    return _state_of(c)


def _append(c, which, new, pos):
    """Row `new` [B, G, D] at token pos[b]: into the tail, and the block into
    the codes when this row completes it."""
    B, G, S, D = c[which].shape
    tail = c[which + "_tail"]
    slot = torch.arange(BLOCK, device="cuda")[None, :] == (pos % BLOCK)[:, None]
    tail.copy_(torch.where(slot[:, None, :, None], new[:, :, None], tail))
    codes, scale = _quantise(tail.float(), c["fmt"])
    done = (pos % BLOCK == BLOCK - 1)[:, None]
    blk, b = (pos // BLOCK).long(), torch.arange(B, device="cuda")
    old = c[which].view(torch.int8).view(B, G, S // BLOCK, BLOCK, D)
    old[b, :, blk] = torch.where(done[..., None, None], codes.view(torch.int8), old[b, :, blk])
    sc = c[which + "_scale"]
    sc[b, :, blk] = torch.where(done, scale, sc[b, :, blk])


def _plain_attend(s):
    case, c, pos = s["case"], s["cache"], s["n"]
    B, G, D, H = case["B"], case["G"], case["D"], case["H"]
    _append(c, "k", s["k_new"], pos)
    _append(c, "v", s["v_new"], pos)
    S = c["k"].shape[2]
    live = torch.arange(S, device="cuda")[None, :] <= pos[:, None]
    scores = s["q"].float().view(B, G, H // G, D) @ _rows(c, "k", pos + 1).transpose(2, 3) * _scale_of(D)
    scores = torch.where(live[:, None, None], scores, torch.full_like(scores, -math.inf))
    e = torch.exp(scores - scores.amax(-1, keepdim=True))
    p = e / e.sum(-1, keepdim=True)
    v = torch.where(live[:, None, :, None], _rows(c, "v", pos + 1), torch.zeros((), device="cuda"))
    s["out"].copy_((p @ v).view(B, H, D))
    if s["weights"] is not None:
        w, add = s["weights"], p.sum(2)
        newest = torch.arange(S, device="cuda")[None, :] == pos[:, None]
        old = torch.where(newest[:, None], torch.zeros_like(w), w)
        w.copy_(torch.where(live[:, None], old + add, w))
    return {"out": s["out"], "weights": s["weights"], "cache": _state_of(c)}


def _plain_sums(s):
    case, n = s["case"], s["n"]
    B, G, D, H, S, W = (case[x] for x in ("B", "G", "D", "H", "S", "W"))
    i = n[:, None] - W + torch.arange(W, device="cuda")[None, :]                      # [B, W] query positions
    rows = torch.gather(s["q"], 1, i.clamp(min=0).long()[:, :, None, None].expand(B, W, H, D))
    q = rows.float().view(B, W, G, H // G, D).permute(0, 2, 3, 1, 4)                   # [B, G, H/G, W, D]
    x = q @ s["k"].float().permute(0, 2, 3, 1)[:, :, None] * _scale_of(D)              # [B, G, H/G, W, S]
    sees = torch.arange(S, device="cuda")[None, None, :] <= i.clamp(min=0)[:, :, None]
    x = torch.where(sees[:, None, None], x, torch.full((), -math.inf, device="cuda"))
    x = torch.exp(x - x.amax(-1, keepdim=True))
    x = x / x.sum(-1, keepdim=True)
    x = torch.where((i >= 0)[:, None, None, :, None], x, torch.zeros((), device="cuda"))
    w = s["weights"][:, :, :S]
    live = torch.arange(S, device="cuda")[None, :] < n[:, None]
    w.copy_(torch.where(live[:, None], x.sum((2, 3)), w))
    return {"weights": s["weights"]}


def _plain_evict(s):
    case, c, n = s["case"], s["cache"], s["n"]
    B, G, D, keep, recent = (case[x] for x in ("B", "G", "D", "keep", "recent"))
    S = c["k"].shape[2]
    at = torch.arange(S, device="cuda")[None, :]
    sure = (at < n[:, None]) & ((at >= n[:, None] - recent) | (n[:, None] <= keep))
    key = torch.where(sure[:, None], torch.full((), math.inf, device="cuda"), s["weights"])
    key = torch.where((at < n[:, None])[:, None], key, torch.full((), -math.inf, device="cuda"))
    first = torch.sort(key, dim=-1, descending=True, stable=True).indices[..., :keep]
    kept = torch.sort(first, -1).values
    m = torch.minimum(n, torch.full_like(n, keep))
    valid = (torch.arange(keep, device="cuda")[None, :] < m[:, None])[:, None]
    s["kept"].copy_(torch.where(valid, kept, torch.full_like(kept, -1)))
    to = s["to"]
    S2 = to["k"].shape[2]
    pad = torch.zeros((B, G, S2 - keep, D), device="cuda")
    at = kept[..., None].expand(B, G, keep, D)
    _set_rows(to, "k", torch.cat([torch.gather(_rows(c, "k", n), 2, at), pad], 2), m)
    _set_rows(to, "v", torch.cat([torch.gather(_rows(c, "v", n), 2, at), pad], 2), m)
    w = s["weights_to"][:, :, :keep]
    w.copy_(torch.where(valid, torch.gather(s["weights"], 2, kept), w))
    s["n_to"].copy_(m)
    return {"kept": s["kept"], "n": s["n_to"], "weights": s["weights_to"], "cache": _state_of(to)}


# -------------------------------------------------------------------- work --

def work(case):
    B, G, D, op = case["B"], case["G"], case["D"], case["op"]
    n = _lens(case)
    tokens = sum(n)
    if op == "store":
        return {"bytes": tokens * G * D * (2 * 2 + 2), "flops": 0}
    if op == "attend":
        H = case["H"]
        b = tokens * G * (2 * D + 8 / BLOCK) + 2 * B * G * D * 4 + 2 * B * H * D * 2
        if case["weights"]:
            b += tokens * G * 8
        return {"bytes": b, "flops": 4 * tokens * H * D}
    if op == "sums":
        H, W = case["H"], case["W"]
        pairs = sum(sum(range(max(0, x - W) + 1, x + 1)) for x in n)
        rows = sum(min(W, x) for x in n)
        return {"bytes": 2 * D * (rows * H + tokens * G) + 4 * tokens * G, "flops": 2 * D * H * pairs}
    m = sum(min(case["keep"], x) for x in n)
    return {"bytes": 4 * tokens * G + m * G * (2 * 2 * D + 4 + 4 + 16 / BLOCK), "flops": 0}


# ------------------------------------------------------------------- exact --
# From the definitions, in float64 and one head at a time.

def _code_of(rows, fmt):
    """Codes (as float64 numbers) and scale of one block [64, D] float64."""
    amax = float(rows.abs().max())
    e = -100
    if amax > 0:
        e = max(-100, math.frexp(amax)[1] - 10)
        e += next(i for i in range(12) if amax <= LIMIT[fmt] * 2.0 ** (e + i))
    y = rows / 2.0 ** e
    if fmt == "int8":
        return torch.round(y), 2.0 ** e
    # e4m3: three bits after the leading one, exponents from -6
    step = torch.exp2(torch.floor(torch.log2(y.abs().clamp(min=2.0 ** -6))) - 3)
    return torch.round(y / step) * step, 2.0 ** e


def _exact_store_head(c, which, b, g, rows, n):
    """Put n rows [n, D] float64 of one head into the float64 copy c."""
    for blk in range(n // BLOCK):
        codes, scale = _code_of(rows[blk * BLOCK:(blk + 1) * BLOCK], c["fmt"])
        c[which][b, g, blk * BLOCK:(blk + 1) * BLOCK] = codes
        c[which + "_scale"][b, g, blk] = scale
    first = (n - 1) // BLOCK * BLOCK
    c[which + "_tail"][b, g, :n - first] = rows[first:n]


def _copy64(c):
    return {k: (v if k == "fmt" else v.double()) for k, v in c.items()}


def _shown(c):
    """The float64 copy as run's outputs; int8 codes are whole numbers."""
    out = {k: v for k, v in c.items() if k != "fmt"}
    if c["fmt"] == "int8":
        out["k"] = out["v"] = None
    return out


def _head_rows(c, which, b, g, n):
    """The n cached rows of one head, float64 [n, D]."""
    S = c[which].shape[2]
    scale = c[which + "_scale"][b, g].double().repeat_interleave(BLOCK)[:S, None]
    x = c[which][b, g].double() * scale
    first = (n - 1) // BLOCK * BLOCK
    return torch.cat([x[:first], c[which + "_tail"][b, g, :n - first].double()])


def exact(case, seed):
    B, G, D, op = case["B"], case["G"], case["D"], case["op"]
    n = _lens(case)
    blocks = B * G * max(case.get("S", 0), min(case.get("N", 0), case.get("keep", 0))) // BLOCK
    if op in ("store", "evict") and blocks > 30000:
        return None
    s = prepare(case, seed)
    if op == "store":
        c = _copy64(s["cache"])
        for b in range(B):
            for g in range(G):
                for w in ("k", "v"):
                    _exact_store_head(c, w, b, g, s[w][b, :n[b], g].double(), n[b])
        return _shown(c)
    scale = 1.0 / math.sqrt(D)
    if op == "attend":
        H, c = case["H"], s["cache"]
        out = torch.empty((B, H, D), dtype=torch.float64, device="cuda")
        weights = None if s["weights"] is None else s["weights"].double()
        after = {w + x: c[w + x].double() for w in ("k", "v") for x in ("_scale", "_tail")}
        codes = {w: None if case["fmt"] == "int8" else c[w].double() for w in ("k", "v")}
        for b in range(B):
            for g in range(G):
                rows = {}
                for w in ("k", "v"):
                    # the rows before the new one: whole blocks as stored, then the tail
                    first = n[b] // BLOCK * BLOCK
                    rows[w] = torch.cat([_head_rows(c, w, b, g, first + BLOCK)[:first],
                                         c[w + "_tail"][b, g, :n[b] - first].double(),
                                         s[w + "_new"][b, g][None].double()])
                    after[w + "_tail"][b, g, n[b] - first] = rows[w][-1]
                    if n[b] - first == BLOCK - 1:
                        code, after[w + "_scale"][b, g, n[b] // BLOCK] = _code_of(rows[w][first:], case["fmt"])
                        if codes[w] is not None:
                            codes[w][b, g, first:first + BLOCK] = code
                hs = slice(g * (H // G), (g + 1) * (H // G))
                p = torch.softmax(s["q"][b, hs].double() @ rows["k"].T * scale, -1)
                out[b, hs] = p @ rows["v"]
                if weights is not None:
                    weights[b, g, n[b]] = 0
                    weights[b, g, :n[b] + 1] += p.sum(0)
        return {"out": out, "weights": weights, "cache": {**codes, **after}}
    if op == "sums":
        H, W = case["H"], case["W"]
        weights = s["weights"].double()
        for b in range(B):
            lo = max(0, n[b] - W)
            hidden = torch.arange(n[b], device="cuda")[None, :] > torch.arange(lo, n[b], device="cuda")[:, None]
            for g in range(G):
                total = 0
                for h in range(g * (H // G), (g + 1) * (H // G)):
                    x = s["q"][b, lo:n[b], h].double() @ s["k"][b, :n[b], g].double().T * scale
                    total = total + torch.softmax(x.masked_fill(hidden, -math.inf), -1).sum(0)
                weights[b, g, :n[b]] = total
        return {"weights": weights}
    c, to = s["cache"], _copy64(s["to"])
    weights, kept = s["weights_to"].double(), torch.full_like(s["kept"], -1)
    for b in range(B):
        m = min(n[b], case["keep"])
        for g in range(G):
            w = s["weights"][b, g].double()
            old = n[b] - min(case["recent"], n[b]) if n[b] > case["keep"] else 0
            heavy = torch.sort(-w[:old], dim=0, stable=True).indices[:m - (n[b] - old)]
            keep = torch.cat([torch.sort(heavy).values, torch.arange(old, n[b], device="cuda")])
            kept[b, g, :m] = keep.to(torch.int32)
            weights[b, g, :m] = w[keep]
            for x in ("k", "v"):
                _exact_store_head(to, x, b, g, _head_rows(c, x, b, g, n[b])[keep], m)
    return {"kept": kept, "n": torch.tensor([min(x, case["keep"]) for x in n], dtype=torch.int32), "weights": weights,
            "cache": _shown(to)}
