"""Cases, plain forms and exact values of the selected-block attention operators.

The operators: rotary positions of q and k (``rotary``), the mean key of every key block and
the blocks that a cheap score selects for each query (``key_means``, ``select_blocks``),
softmax attention over the selected blocks with its backward pass (``selected_attn``,
``selected_attn_backward``), and the three last for single tokens over a key / value cache.

Definitions, per batch element and key / value head (the G = heads / kv_heads query heads of
a group share one selection):

  mean    m_g = sum_{j in block g, j < kv_len} k_j / (number of such j), held in 32 bits
  score   s_ig = (sum_{h in group} q_ih) . m_g
  select  among the blocks with a key below kv_len (causal: and at or before the query's
          position p_i = q_start + i): the first n_first, the query's own and the n_local - 1
          before it (causal only), then the largest scores, ties to the lower block, ``top``
          in all, ascending, -1 where there are fewer
  attend  softmax over the keys j of the selected blocks, j < kv_len (causal: j <= p_i);
          a query without keys gives a zero row and a log-sum-exp of -inf
  rotary  pair (a, b) of the rotated part at position p: f (a cos t - b sin t,
          b cos t + a sin t), t = p * freq of the pair, f the scaling's factor
"""
import math

import torch

own = False

BF16, F32 = "bf16", "f32"
_TYPE = {BF16: torch.bfloat16, F32: torch.float32}


def _rotary(name, dtype, batch, heads, kv_heads, tokens, d, rot, layout, axes, scaling, far, inverse, token_major):
    return {"name": name, "kind": "rotary", "dtype": dtype, "batch": batch, "heads": heads, "kv_heads": kv_heads,
            "tokens": tokens, "d": d, "rot": rot, "layout": layout, "axes": axes, "scaling": scaling, "far": far,
            "inverse": inverse, "token_major": token_major}


def _blocks(name, kind, dtype, batch, heads, kv_heads, tokens, keys, d, block, top, causal, first, local, ragged):
    return {"name": name, "kind": kind, "dtype": dtype, "batch": batch, "heads": heads, "kv_heads": kv_heads,
            "tokens": tokens, "keys": keys, "d": d, "block": block, "top": top, "causal": causal, "first": first,
            "local": local, "ragged": ragged}


def listed():
    return [
        # the rotation of one new token of each of eight sequences far into a long, scaled context
        _rotary("rotary-token-step", BF16, 8, 32, 8, 1, 128, 128, "half", 1, "ramp", 131072, False, True),
        # q and k of the 40-head, 75,600-token video call: three position axes (t, y, x), interleaved pairs
        _rotary("rotary-video", BF16, 1, 40, 40, 75600, 128, 128, "interleaved", 3, "none", 0, False, False),
        # the gradient's rotation in training: half of each head rotated, token-major projections, grouped heads
        _rotary("rotary-grad-partial", BF16, 2, 16, 4, 32760, 128, 64, "half", 1, "linear", 0, True, True),
        # selection for the 8-head, 8,192-token workload (bidirectional, as in a video transformer)
        _blocks("select-small", "select", BF16, 1, 8, 8, 8192, 8192, 128, 128, 12, False, 0, 0, False),
        # selection in a causal grouped-head prompt, odd length, one padded sequence, first and local blocks kept
        _blocks("select-causal-grouped", "select", BF16, 2, 32, 8, 16383, 16383, 128, 128, 16, True, 1, 2, True),
        # attention in 32 bits on the smallest workload of the repository
        _blocks("attend-tiny-f32", "attend", F32, 1, 2, 2, 1024, 1024, 64, 64, 4, False, 0, 0, False),
        # the 16-head, 32,760-token workload: 16 of its 256 blocks for each query (the last block is short)
        _blocks("attend-broad", "attend", BF16, 1, 16, 16, 32760, 32760, 128, 128, 16, False, 0, 0, False),
        # a causal grouped-head prompt of odd length with one padded sequence
        _blocks("attend-causal-grouped", "attend", BF16, 2, 32, 8, 8191, 8191, 128, 64, 16, True, 1, 2, True),
        # a small training step in 32 bits, ragged length
        _blocks("train-tiny-f32", "train", F32, 1, 2, 2, 1000, 1000, 64, 64, 4, True, 0, 1, False),
        # a training step (forward and backward) of the 16-head workload at a quarter of its selection
        _blocks("train-broad", "train", BF16, 1, 16, 16, 32760, 32760, 128, 128, 8, False, 0, 0, False),
        # one token of one sequence over a cache: latency
        _blocks("decode-one", "decode", BF16, 1, 32, 8, 1, 8192, 128, 128, 16, True, 1, 2, True),
        # one token of each of 32 sequences of different lengths over a long cache
        _blocks("decode-batch", "decode", BF16, 32, 32, 8, 1, 32768, 128, 64, 32, True, 1, 2, True),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    """One more case of the listed ranges: both types and head sizes, grouped and plain heads, odd lengths."""
    most = {}
    for c in listed():
        for what, x in _cost(c).items():
            most[what] = max(most.get(what, 0), x)
    c = _drawn(rng)
    while any(x > most[what] for what, x in _cost(c).items()):  # no dearer than the largest listed case
        c["tokens"] = c["tokens"] * 2 // 3
        if "keys" in c:
            c["keys"] = c["keys"] * 2 // 3 if c["kind"] == "decode" else c["tokens"]
            c["tokens"] = 1 if c["kind"] == "decode" else c["tokens"]
    return c


def _cost(c):
    """Work of a case and, for attention, what its plain form multiplies: whole rows, not only the selected blocks."""
    whole = {"attend": 1, "train": 4}.get(c["kind"], 0) * c["batch"] * c["heads"] * c["tokens"] * c.get("keys", 0)
    return {**work(c), "whole": whole * c["d"]}


def _drawn(rng):
    kind = rng.choice(["rotary", "select", "attend", "attend", "train", "decode"])
    dtype = F32 if rng.random() < 0.2 else BF16
    d, block = rng.choice([64, 128]), rng.choice([64, 128])
    kv_heads, group = rng.choice([1, 2, 4, 8]), rng.choice([1, 1, 2, 3, 4, 8])
    causal = rng.random() < 0.6
    if kind == "rotary":
        batch, tokens = rng.randint(1, 4), _log(rng, 1, 20000)
        axes = rng.choice([1, 1, 3])
        rot = d if axes == 3 else rng.choice([d, d // 2, 3 * d // 4])
        return _rotary("", dtype, batch, kv_heads * group, kv_heads, tokens, d, rot, rng.choice(["half", "interleaved"]),
                       axes, rng.choice(["none", "linear", "base", "ramp"]), rng.choice([0, 131072]) if axes == 1 else 0,
                       rng.random() < 0.4, rng.random() < 0.5)
    if kind == "decode":
        keys = _log(rng, 300, 32768)
        top = rng.randint(4, 32)
        return _blocks("", kind, dtype, _log(rng, 1, 24), kv_heads * group, kv_heads, 1, keys, d, block, top, True,
                       rng.randint(0, 2), rng.randint(1, 2), True)
    # attention in 32 bits and training cost the most: shorter
    most = 4096 if dtype == F32 else 12000 if kind == "train" else 16000
    tokens = _log(rng, 100, most)
    batch = rng.randint(1, 2)
    return _blocks("", kind, dtype, batch, kv_heads * group, kv_heads, tokens, tokens, d, block, rng.randint(3, 24), causal,
                   rng.randint(0, 1) if causal else 0, rng.randint(1, 2) if causal else 0, rng.random() < 0.5)


# ------------------------------------------------------------------------------- inputs

def _latent(gen, batch, tokens, d, dev):
    """Token latents: smooth position features, a mean that runs of tokens share, and noise."""
    t = torch.arange(tokens, device=dev, dtype=torch.float32) / max(tokens, 64)
    feats = torch.stack([f(2 * math.pi * 2.0 ** i * t) for i in range(4) for f in (torch.sin, torch.cos)], -1)
    w = torch.randn(8, d, generator=gen, device=dev) / math.sqrt(8)
    means = torch.randn(batch, 64, d, generator=gen, device=dev)
    runs = torch.randint(0, 64, (batch, tokens // 48 + 1), generator=gen, device=dev).repeat_interleave(48, 1)[:, :tokens]
    x = 0.5 * torch.randn(batch, tokens, d, generator=gen, device=dev)
    x += feats @ w
    x += torch.gather(means, 1, runs[..., None].expand(-1, -1, d))
    return x


def _project(gen, x, heads, dtype):
    """[batch, heads, tokens, d] projections of the latents, a Gaussian matrix for each head."""
    b, n, d = x.shape
    out = torch.empty(b, heads, n, d, device=x.device, dtype=dtype)
    for h in range(heads):
        w = torch.randn(d, d, generator=gen, device=x.device) / math.sqrt(d)
        out[:, h] = (x @ w).to(dtype)
    return out


def _positions(case, gen, dev):
    b, n, axes = case["batch"], case["tokens"], case["axes"]
    if axes == 3:  # raster order of a (t, y, x) grid, rows of 80 and planes of 45 rows as in the video call
        i = torch.arange(n, device=dev)
        return torch.stack([i // 3600, i // 80 % 45, i % 80], -1).int().expand(b, n, 3).contiguous()
    start = torch.randint(0, max(1, case["far"] - n), (b, 1), generator=gen, device=dev) if case["far"] else \
        torch.zeros(b, 1, device=dev, dtype=torch.int64)
    return (start + torch.arange(n, device=dev)[None]).int()[..., None].contiguous()


def _sections(case):
    pairs = case["rot"] // 2
    return [pairs] if case["axes"] == 1 else [pairs - 2 * (pairs // 3), pairs // 3, pairs // 3]


_BASE, _FACTOR, _TRAINED = 10000.0, 8.0, 16384


def _frequencies(case):
    """([pairs] radians for each step of the position, factor): 64-bit, on the host."""
    freqs, factor = [], 1.0
    for p in _sections(case):
        base = _BASE
        if case["scaling"] == "base":
            base = base * _FACTOR ** (2 * p / (2 * p - 2))
        f = [base ** (-i / p) for i in range(p)]
        if case["scaling"] == "linear":
            f = [x / _FACTOR for x in f]
        if case["scaling"] == "ramp":  # few turns within the trained length: interpolated; many: kept
            keep = [min(1.0, max(0.0, (_TRAINED * x / (2 * math.pi) - 1.0) / 31.0)) for x in f]
            f = [x * g + x / _FACTOR * (1.0 - g) for x, g in zip(f, keep)]
            factor = 0.1 * math.log(_FACTOR) + 1.0
        freqs += f
    return freqs, factor


def _pick(case, q, k, lens):
    """Selected blocks from products in 64 bits (the inputs of the attention cases)."""
    means = _plain_means(k, case["block"], lens)
    return _plain_select(case, q, means, lens, _starts(case, lens))


def _starts(case, lens):
    """Position of query 0: a new token sits at the end of its sequence, a prompt starts at 0."""
    return lens - 1 if case["kind"] == "decode" else torch.zeros_like(lens)


def prepare(case, seed):
    dev = torch.device("cuda")
    gen = torch.Generator(device=dev)
    gen.manual_seed(seed)
    dt = _TYPE[case["dtype"]]
    b, hq, hk, n, d = case["batch"], case["heads"], case["kv_heads"], case["tokens"], case["d"]
    s = {"case": case}
    if own:
        import free_block_sparse_response_b200 as spr
        s["spr"] = spr
    if case["kind"] == "rotary":
        for name, h in (("q", hq), ("k", hk)):
            x = torch.randn(b, n, h, d, generator=gen, device=dev).to(dt)
            s[name] = x.transpose(1, 2) if case["token_major"] else x.view(b, h, n, d)
        s["positions"] = _positions(case, gen, dev)
        freqs, s["factor"] = _frequencies(case)
        s["freqs"] = torch.tensor(freqs, dtype=torch.float64, device=dev)
        if own:
            s["plan"] = spr.rotary_plan(d, dev, rot_dim=case["rot"], sections=_sections(case), base=_BASE,
                                        layout={"half": spr.ROTARY_HALF, "interleaved": spr.ROTARY_INTERLEAVED}[case["layout"]],
                                        scaling=case["scaling"], scaling_factor=_FACTOR, trained_length=_TRAINED)
        return s
    keys = case["keys"]
    x = _latent(gen, b, keys, d, dev)
    s["k"], s["v"] = _project(gen, x, hk, dt), _project(gen, x, hk, dt)
    s["q"] = _project(gen, x[:, keys - n:], hq, dt)
    del x
    lens = torch.full((b,), keys, dtype=torch.int32, device=dev)
    if case["ragged"]:
        low = max(1, keys // 3)
        lens = torch.randint(low, keys + 1, (b,), generator=gen, device=dev, dtype=torch.int32)
        if case["kind"] != "decode":
            lens[0] = keys
    s["lens"], s["starts"] = lens, _starts(case, lens).int()
    if case["kind"] in ("attend", "train"):
        s["sel"] = _pick(case, s["q"], s["k"], lens)
    if case["kind"] == "train":
        s["grad"] = torch.randn(b, hq, n, d, generator=gen, device=dev).to(dt)
    if case["kind"] == "decode":
        s["means"] = _plain_means(s["k"], case["block"], lens - 1)  # the cache's means, kept up to the token before
    if own:
        s["cfg"] = spr.SelectConfig(block=case["block"], top=case["top"], causal=case["causal"], n_first=case["first"],
                                    n_local=case["local"])
        s["ws"] = spr.selected_workspace(s["q"], s["k"], s["cfg"], backward=case["kind"] == "train")
    return s


# ------------------------------------------------------------------- the plain form and own

def run(state):
    return {"rotary": _run_rotary, "select": _run_select, "attend": _run_attend, "train": _run_train,
            "decode": _run_decode}[state["case"]["kind"]](state)


def _run_rotary(s):
    c = s["case"]
    if own:
        q, k = s["spr"].rotary(s["plan"], s["positions"], s["q"], s["k"], inverse=c["inverse"])
        return {"q": q, "k": k}
    return {"q": _plain_rotary(s, s["q"]), "k": _plain_rotary(s, s["k"])}


def _run_select(s):
    if own:
        means = s["spr"].key_means(s["k"], s["cfg"].block, kv_len=s["lens"])
        sel = s["spr"].select_blocks(s["q"], means, s["k"].shape[2], s["cfg"], s["ws"], kv_len=s["lens"], q_start=s["starts"])
        return {"means": means, "sel": sel}
    means = _plain_means(s["k"], s["case"]["block"], s["lens"])
    return {"means": means, "sel": _plain_select(s["case"], s["q"], means, s["lens"], s["starts"])}


def _run_attend(s):
    if own:
        out, lse = s["spr"].selected_attn(s["q"], s["k"], s["v"], s["sel"], s["cfg"], s["ws"], kv_len=s["lens"],
                                          q_start=s["starts"])
    else:
        out, lse = _plain_attend(s["case"], s["q"], s["k"], s["v"], s["sel"], s["lens"], s["starts"])
    return {"out": out, "lse": lse}


def _run_train(s):
    if own:  # bf16: with what the rounding of out left off, which dq needs
        q = s["q"]
        rest = torch.empty(q.shape, dtype=q.dtype, device=q.device) if q.dtype == torch.bfloat16 else None
        out, lse = s["spr"].selected_attn(q, s["k"], s["v"], s["sel"], s["cfg"], s["ws"], kv_len=s["lens"],
                                          q_start=s["starts"], rest=rest)
        dq, dk, dv = s["spr"].selected_attn_backward(s["grad"], q, s["k"], s["v"], out, lse, s["sel"], s["cfg"],
                                                     s["ws"], kv_len=s["lens"], q_start=s["starts"], rest=rest)
    else:
        out, dq, dk, dv = _plain_train(s["case"], s["q"], s["k"], s["v"], s["sel"], s["lens"], s["starts"], s["grad"])
    return {"out": out, "dq": dq, "dk": dk, "dv": dv}


def _run_decode(s):
    c = s["case"]
    if own:  # the new key's block, the selection, the attention
        spr = s["spr"]
        spr.key_means(s["k"], c["block"], kv_len=s["lens"], kv_start=s["starts"], max_new=1, out=s["means"])
        sel = spr.select_blocks(s["q"], s["means"], s["k"].shape[2], s["cfg"], s["ws"], kv_len=s["lens"], q_start=s["starts"])
        out, _ = spr.selected_attn(s["q"], s["k"], s["v"], sel, s["cfg"], s["ws"], kv_len=s["lens"], q_start=s["starts"])
        return {"out": out, "sel": sel, "means": s["means"]}
    b, hk, nk, d = s["k"].shape
    blk = c["block"]
    g = (s["lens"].long() - 1) // blk
    j = torch.arange(blk, device=g.device)
    at = (g[:, None] * blk + j[None]).clamp(max=nk - 1)
    live = g[:, None] * blk + j[None] < s["lens"][:, None]
    rows = torch.gather(s["k"], 2, at[:, None, :, None].expand(b, hk, blk, d)).double()
    m = torch.where(live[:, None, :, None], rows, 0.0).sum(2) / live.sum(1)[:, None, None]
    s["means"].scatter_(2, g[:, None, None, None].expand(b, hk, 1, d), m[:, :, None].float())
    sel = _plain_select(c, s["q"], s["means"], s["lens"], s["starts"])
    # gather the selected blocks of the cache: [b, hk, top * block, d]
    grp = c["heads"] // hk
    idx = (sel[:, :, 0].clamp(min=0).long()[..., None] * blk + j).flatten(2)
    pos = idx
    ok = (sel[:, :, 0] >= 0)[..., None].expand(b, hk, c["top"], blk).flatten(2) & (pos < s["lens"][:, None, None])
    idx = idx.clamp(max=nk - 1)[..., None].expand(-1, -1, -1, d)
    kk, vv = torch.gather(s["k"], 2, idx).float(), torch.gather(s["v"], 2, idx).float()
    x = torch.einsum("bhgd,bhjd->bhgj", s["q"].view(b, hk, grp, d).float(), kk) / math.sqrt(d)
    x = torch.where(ok[:, :, None], x, -math.inf)
    e = torch.exp(x - x.amax(-1, keepdim=True))
    e = torch.where(ok[:, :, None], e, 0.0)
    out = torch.einsum("bhgj,bhjd->bhgd", e / e.sum(-1, keepdim=True), torch.where(ok[..., None], vv, 0.0))
    return {"out": out.reshape(b, c["heads"], 1, d).to(s["q"].dtype), "sel": sel, "means": s["means"]}


def _plain_rotary(s, x):
    c = s["case"]
    r, pairs = c["rot"], c["rot"] // 2
    axis = torch.tensor([a for a, p in enumerate(_sections(c)) for _ in range(p)], device=x.device)
    t = s["positions"].double()[..., axis] * s["freqs"]  # [b, n, pairs]: far positions need 64 bits
    cos, sin = (s["factor"] * torch.cos(t)).float()[:, None], (s["factor"] * torch.sin(t)).float()[:, None]
    if c["inverse"]:
        sin = -sin
    out = torch.empty_like(x)
    some = max(1, (1 << 26) // (x.shape[0] * x.shape[2] * x.shape[3]))  # heads at a time: 32 bits of the largest call
    for h in range(0, x.shape[1], some):
        xf = x[:, h:h + some].float()
        if c["layout"] == "half":
            a, b2 = xf[..., :pairs], xf[..., pairs:r]
            y = torch.cat([a * cos - b2 * sin, b2 * cos + a * sin, xf[..., r:]], -1)
        else:
            a, b2 = xf[..., 0:r:2], xf[..., 1:r:2]
            y = torch.cat([torch.stack([a * cos - b2 * sin, b2 * cos + a * sin], -1).flatten(-2), xf[..., r:]], -1)
        out[:, h:h + some] = y.to(x.dtype)
    return out


def _plain_means(k, block, lens):
    b, hk, n, d = k.shape
    g = -(-n // block)
    means = torch.empty(b, hk, g, d, device=k.device)
    live = torch.arange(g * block, device=k.device)[None] < lens[:, None]  # [b, g * block]
    cnt = live.view(b, 1, g, block).sum(-1).clamp(min=1)
    some = max(1, (1 << 28) // (b * g * block * d))
    for h in range(0, hk, some):
        x = torch.nn.functional.pad(k[:, h:h + some].double(), (0, 0, 0, g * block - n))
        x = torch.where(live[:, None, :, None], x, 0.0).unflatten(2, (g, block)).sum(3)
        means[:, h:h + some] = (x / cnt[..., None]).float()
    return means


def _plain_select(c, q, means, lens, starts):
    b, hq, n, d = q.shape
    hk, g = means.shape[1], means.shape[2]
    top, blk = c["top"], c["block"]
    ids = torch.arange(g, device=q.device)
    sel = torch.full((b, hk, n, top), -1, dtype=torch.int32, device=q.device)
    mt = means.double().transpose(2, 3)
    rows = max(1, (1 << 26) // (g * b * hk))
    for r in range(0, n, rows):
        qs = q[:, :, r:r + rows].unflatten(1, (hk, hq // hk)).double().sum(2)
        sc = qs @ mt  # 64 bits: values next to the border of the selection
        ok = (ids * blk < lens[:, None])[:, None, None]  # [b, 1, 1, g]
        forced = ids < c["first"]
        if c["causal"]:
            p = starts.long()[:, None] + torch.arange(r, r + sc.shape[2], device=q.device)
            mine = torch.div(p, blk, rounding_mode="floor")[:, None, :, None]
            ok = ok & (ids * blk <= p[:, None, :, None])
            forced = forced | ((ids <= mine) & (ids > mine - c["local"]))
        sc = torch.where(ok, torch.where(forced, math.inf, sc), -math.inf)
        at = torch.sort(sc, dim=-1, descending=True, stable=True).indices[..., :top]  # ties: the lower block
        at = torch.where(torch.gather(ok.expand(sc.shape), 3, at), at, g)
        at = torch.sort(at, dim=-1).values
        sel[:, :, r:r + rows, :at.shape[-1]] = torch.where(at < g, at, -1).int()
    return sel


def _mask(c, sel, r, rows, keys, length, start):
    """[rows, keys]: the keys that rows r .. of one (batch, key / value head) attend to."""
    g = -(-keys // c["block"])
    at = sel[r:r + rows].long()
    m = torch.zeros(at.shape[0], g + 1, dtype=torch.bool, device=sel.device)
    m.scatter_(1, torch.where(at >= 0, at, g), True)
    m = m[:, :g].repeat_interleave(c["block"], 1)[:, :keys]
    j = torch.arange(keys, device=sel.device)
    m = m & (j < length)[None]
    if c["causal"]:
        m = m & (j[None] <= start + torch.arange(r, r + at.shape[0], device=sel.device)[:, None])
    return m


def _plain_attend(c, q, k, v, sel, lens, starts):
    b, hq, n, d = q.shape
    hk, keys = k.shape[1], k.shape[2]
    out = torch.zeros_like(q)
    lse = torch.empty(b, hq, n, device=q.device)
    rows = max(1, (1 << 28) // keys)
    for i in range(b):
        for h in range(hq):
            kh = h // (hq // hk)
            kf, vf = k[i, kh].float(), v[i, kh].float()
            for r in range(0, n, rows):
                x = q[i, h, r:r + rows].float() @ kf.t()
                x *= 1.0 / math.sqrt(d)
                x.masked_fill_(~_mask(c, sel[i, kh], r, rows, keys, lens[i], starts[i]), -math.inf)
                top = x.amax(-1, keepdim=True)
                x -= torch.where(top == -math.inf, 0.0, top)
                x.exp_()
                l = x.sum(-1, keepdim=True)
                out[i, h, r:r + rows] = (x @ vf / torch.where(l > 0, l, 1.0)).to(q.dtype)
                lse[i, h, r:r + rows] = (top + torch.log(l))[:, 0]
    return out, lse


def _plain_train(c, q, k, v, sel, lens, starts, grad):
    b, hq, n, d = q.shape
    hk, keys = k.shape[1], k.shape[2]
    scale = 1.0 / math.sqrt(d)
    out, dq = torch.zeros_like(q), torch.zeros_like(q)
    dk, dv = torch.zeros_like(k), torch.zeros_like(v)
    rows = max(1, (1 << 28) // keys)
    for i in range(b):
        for kh in range(hk):
            kf, vf = k[i, kh].float(), v[i, kh].float()
            gk, gv = torch.zeros_like(kf), torch.zeros_like(vf)
            for r in range(0, n, rows):
                hide = ~_mask(c, sel[i, kh], r, rows, keys, lens[i], starts[i])
                for h in range(kh * (hq // hk), (kh + 1) * (hq // hk)):
                    qf, gf = q[i, h, r:r + rows].float(), grad[i, h, r:r + rows].float()
                    p = qf @ kf.t()
                    p *= scale
                    p.masked_fill_(hide, -math.inf)
                    top = p.amax(-1, keepdim=True)
                    p -= torch.where(top == -math.inf, 0.0, top)
                    p.exp_()
                    l = p.sum(-1, keepdim=True)
                    p /= torch.where(l > 0, l, 1.0)
                    of = p @ vf
                    out[i, h, r:r + rows] = of.to(q.dtype)
                    gv += p.t() @ gf
                    ds = gf @ vf.t()
                    ds -= (gf * of).sum(-1, keepdim=True)
                    ds *= p
                    ds *= scale
                    dq[i, h, r:r + rows] = (ds @ kf).to(q.dtype)
                    gk += ds.t() @ qf
            dk[i, kh], dv[i, kh] = gk.to(k.dtype), gv.to(v.dtype)
    return out, dq, dk, dv


# ------------------------------------------------------------------------- exact values

def exact(case, seed):
    """The operators' definitions in 64 bits, written apart from the plain forms above."""
    s = prepare(case, seed)
    kind = case["kind"]
    if kind == "rotary":
        return {"q": _exact_rotary(s, s["q"]), "k": _exact_rotary(s, s["k"])}
    if kind == "select":
        means = _exact_means(case, s["k"], s["lens"])
        return {"means": means, "sel": _exact_select(case, s["q"], means.float(), s["lens"], s["starts"])}
    if kind == "attend":
        out, lse, _ = _exact_attend(case, s["q"], s["k"], s["v"], s["sel"], s["lens"], s["starts"], None)
        return {"out": out, "lse": lse}
    if kind == "train":
        out, _, (dq, dk, dv) = _exact_attend(case, s["q"], s["k"], s["v"], s["sel"], s["lens"], s["starts"], s["grad"])
        return {"out": out, "dq": dq, "dk": dk, "dv": dv}
    means = _exact_means(case, s["k"], s["lens"])
    sel = _exact_select(case, s["q"], means.float(), s["lens"], s["starts"])
    out, _, _ = _exact_attend(case, s["q"], s["k"], s["v"], sel, s["lens"], s["starts"], None)
    return {"out": out, "sel": sel, "means": means}


def _exact_rotary(s, x):
    """Each pair as a complex number times f exp(i t)."""
    c = s["case"]
    r = c["rot"]
    bounds = [0]
    for p in _sections(c):
        bounds.append(bounds[-1] + p)
    t = torch.cat([s["positions"][..., a:a + 1].double() * s["freqs"][bounds[a]:bounds[a + 1]] for a in range(c["axes"])], -1)
    turn = torch.polar(torch.full_like(t, s["factor"]), -t if c["inverse"] else t)
    out = torch.empty(x.shape, dtype=torch.float64, device=x.device)
    for h in range(x.shape[1]):
        y = x[:, h].double()
        z = torch.complex(y[..., :r // 2], y[..., r // 2:r]) if c["layout"] == "half" else \
            torch.view_as_complex(y[..., :r].reshape(*y.shape[:-1], r // 2, 2).contiguous())
        z = z * turn
        out[:, h, :, :r] = torch.cat([z.real, z.imag], -1) if c["layout"] == "half" else torch.view_as_real(z).flatten(-2)
        out[:, h, :, r:] = y[..., r:]
    return out


def _exact_means(c, k, lens):
    b, hk, n, d = k.shape
    out = torch.zeros(b, hk, -(-n // c["block"]), d, dtype=torch.float64, device=k.device)
    for i, m in enumerate(lens.tolist()):
        full = m // c["block"]
        out[i, :, :full] = k[i, :, :full * c["block"]].unflatten(1, (full, c["block"])).mean(2, dtype=torch.float64)
        if m % c["block"]:
            out[i, :, full] = k[i, :, full * c["block"]:m].mean(1, dtype=torch.float64)
    return out


def _exact_select(c, q, means, lens, starts):
    """Rank of each block by counting the blocks that come before it."""
    b, hq, n, d = q.shape
    hk, g = means.shape[1], means.shape[2]
    sel = torch.full((b, hk, n, c["top"]), -1, dtype=torch.int32, device=q.device)
    rows = max(1, (1 << 26) // (g * g))
    blk = torch.arange(g, device=q.device)
    for i, m in enumerate(lens.tolist()):
        for h in range(hk):
            qs = q[i].unflatten(0, (hk, hq // hk))[h].sum(0, dtype=torch.float64)
            for r in range(0, n, rows):
                part = qs[r:r + rows]
                p = int(starts[i]) + torch.arange(r, r + part.shape[0], device=q.device)
                last = torch.minimum(p // c["block"], torch.tensor((m - 1) // c["block"], device=q.device)) if c["causal"] else \
                    torch.full_like(p, (m - 1) // c["block"])
                can = blk[None] <= last[:, None]
                must = (blk < c["first"])[None].expand(can.shape)
                if c["causal"]:
                    mine = (p // c["block"])[:, None]
                    must = must | ((blk[None] <= mine) & (mine - blk[None] < c["local"]))
                score = torch.einsum("nd,gd->ng", part, means[i, h].double())
                score = torch.where(must, math.inf, score)
                score = torch.where(can, score, -math.inf)
                above = (score[:, None, :] > score[:, :, None]) | \
                    ((score[:, None, :] == score[:, :, None]) & (blk[None, None] < blk[None, :, None]))
                taken = can & (above.sum(-1) < c["top"])
                slot = taken.cumsum(-1) - 1
                row, at = taken.nonzero(as_tuple=True)
                sel[i, h, r + row, slot[row, at]] = at.int()
    return sel


def _exact_attend(c, q, k, v, sel, lens, starts, grad):
    """Softmax attention by torch.logsumexp, gradients by automatic differentiation, rows at a time."""
    b, hq, n, d = q.shape
    hk, keys = k.shape[1], k.shape[2]
    out = torch.zeros(q.shape, dtype=torch.float64, device=q.device)
    lse = torch.full(q.shape[:3], -math.inf, dtype=torch.float64, device=q.device)
    dq = dk = dv = None
    if grad is not None:
        dq, dk, dv = (torch.zeros(x.shape, dtype=torch.float64, device=q.device) for x in (q, k, v))
    rows = max(1, (1 << 26) // keys)
    of_key = torch.arange(keys, device=q.device) // c["block"]
    j = torch.arange(keys, device=q.device)
    for i, m in enumerate(lens.tolist()):
        for h in range(hq):
            kh = h // (hq // hk)
            kd, vd = k[i, kh].double(), v[i, kh].double()
            for r in range(0, n, rows):
                at = sel[i, kh, r:r + rows]
                taken = torch.zeros(at.shape[0], int(of_key[-1]) + 1, dtype=torch.int32, device=q.device)
                for t in range(at.shape[1]):
                    taken.scatter_add_(1, at[:, t:t + 1].clamp(min=0).long(), (at[:, t:t + 1] >= 0).int())
                ok = taken[:, of_key] > 0
                ok &= j < m
                if c["causal"]:
                    ok &= j[None] - int(starts[i]) <= torch.arange(r, r + at.shape[0], device=q.device)[:, None]
                has = ok.any(-1)
                qd = q[i, h, r:r + rows].double()
                ins = [t.detach().requires_grad_(grad is not None) for t in (qd, kd, vd)]
                with torch.set_grad_enabled(grad is not None):
                    x = ins[0] @ ins[1].t() * d ** -0.5
                    x = torch.where(ok, x, -1e300)
                    ls = torch.logsumexp(x, -1, keepdim=True)
                    y = torch.where(ok, torch.exp(x - ls), 0.0) @ ins[2]
                    if grad is not None:
                        a = torch.autograd.grad(y, ins, grad[i, h, r:r + rows].double())
                        dq[i, h, r:r + rows] = a[0]
                        dk[i, kh] += a[1]
                        dv[i, kh] += a[2]
                out[i, h, r:r + rows] = y.detach()
                lse[i, h, r:r + rows] = torch.where(has, ls.detach()[:, 0], -math.inf)
    return out, lse, (dq, dk, dv)


# ------------------------------------------------------------------------- the work of a pass

def work(case):
    """Bytes: inputs once, outputs once (a selection's blocks of a cache once). Flops: products of live pairs."""
    c = case
    e = 2 if c["dtype"] == BF16 else 4
    b, hq, hk, n, d = c["batch"], c["heads"], c["kv_heads"], c["tokens"], c["d"]
    if c["kind"] == "rotary":
        x = b * (hq + hk) * n
        return {"bytes": 2 * x * d * e + b * n * c["axes"] * 4, "flops": 3 * x * c["rot"]}
    keys, blk, top = c["keys"], c["block"], c["top"]
    g = -(-keys // blk)
    if c["kind"] == "decode":
        taken = min(top, g) * blk
        return {"bytes": b * (hk * (2 * taken * d * e + g * d * 4) + 2 * hq * d * e + hk * top * 4),
                "flops": b * (4 * hq * taken * d + 2 * hk * g * d)}
    if c["kind"] == "select":
        half = 0.5 if c["causal"] else 1.0
        return {"bytes": b * (hq * n * d * e + hk * keys * d * e + hk * g * d * 4 + hk * n * top * 4),
                "flops": b * hk * (n * g * d * 2 * half + keys * d)}
    # a query's selected blocks: fewer at the start of a causal prompt
    if c["causal"]:
        pairs = sum(min(top, i // blk + 1) * blk - (blk - 1 - i % blk) for i in range(n))
    else:
        pairs = n * min(top, g) * blk
    io = hq * n * d * e + 2 * hk * keys * d * e + hk * n * top * 4 + hq * n * d * e + hq * n * 4
    flops = 4 * d * pairs * hq
    if c["kind"] == "train":
        io += 2 * hq * n * d * e + 2 * hk * keys * d * e
        flops += 10 * d * pairs * hq
    return {"bytes": b * io, "flops": b * flops}
