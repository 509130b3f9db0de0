"""What is measured of the operators around a block's attention: the norm and rotation of queries and
keys, attention over a sliding window with first tokens that stay visible, and attention of a batch
that shares a prefix.

`run` computes them in their plain form (elementary torch operations in 32 bits, rounded once),
or, where `own` is true, through the library's entry points.  Inputs are bf16, the rotation's tables
float32; packed batches carry their row offsets `cu` [batch + 1] on the GPU, as the calls take them.
"""
import math

import numpy as np
import torch

own = False

# A serving program keeps one workspace for all its layers; 64 MiB is also what the library's
# allocation-free forward holds.
WORKSPACE = 64 << 20


# ------------------------------------------------------------------ cases
def _rope(name, rows, hq, hk, d, rot, pairs, norm, bias, table, given, fused):
    """rows: the lengths of the sequences; rot: channels of a head that are rotated; pairs: neighbours
    (2i, 2i + 1) or halves (i, i + rot / 2); table: positions it has; given: the tokens' positions come
    in a tensor (else a token's number in its sequence); fused: Q and K are column slices of one
    [tokens, (hq + 2 hk) d] projection output."""
    return dict(name=name, op="rope", rows=rows, hq=hq, hk=hk, d=d, rot=rot, pairs=pairs, norm=norm, bias=bias,
                table=table, given=given, fused=fused)


def _window(name, q, k, hq, hkv, d, causal, left, right, sinks, lse=False, fused=False):
    """q, k: the lengths of the sequences, comma separated; left, right: keys before and behind the
    query's own that it sees (-1: all of them); sinks: first keys that stay visible."""
    return dict(name=name, op="window", q=q, k=k, hq=hq, hkv=hkv, d=d, causal=causal, left=left, right=right,
                sinks=sinks, lse=lse, fused=fused)


def _prefix(name, prefix, q, k, hq, hkv, d, causal, lse=False):
    """prefix: keys that all sequences share; q, k: the sequences' own lengths."""
    return dict(name=name, op="prefix", prefix=prefix, q=q, k=k, hq=hq, hkv=hkv, d=d, causal=causal, lse=lse)


def listed():
    return [
        # one new token for each of 16 sequences at far positions, shared key heads: latency
        _rope("rope_tokens_16", ",".join(["1"] * 16), 32, 8, 128, 128, "halves", "rms", False, 131072, True, True),
        # the joint attention of a DiT block (4608 tokens, 24 heads of 128), out of the fused QKV projection
        _rope("rope_dit_block", "4608", 24, 24, 128, 128, "neighbours", "rms", False, 4608, True, True),
        # packed images and their prompts: LayerNorm with bias, part of each head rotated
        _rope("rope_packed_layer", "77,4099,1,9001,154,2500", 16, 16, 72, 40, "halves", "layer", True, 9001, False, False),
        # a text encoder's local layer on one prompt: latency is all there is
        _window("window_prompt_77", "77", "77", 10, 10, 64, True, 31, 0, 1, fused=True),
        # one new token for each of 16 sequences against long, unequal histories: window and first tokens
        _window("window_one_token", ",".join(["1"] * 16),
                "8192,517,4096,1,2049,7777,63,3000,6143,129,1024,5000,2500,8000,64,900", 32, 8, 128, True, 1023, 0, 4,
                lse=True),
        # prompts of different lengths packed behind each other, causal, shared key heads
        _window("window_packed_prompts", "1,17,511,2048,1023,4096,333,6400", "1,17,511,2048,1023,4096,333,6400",
                32, 8, 128, True, 511, 0, 4, lse=True),
        # a long video's tokens: each sees its neighbours on both sides, and the prompt's tokens in front
        _window("window_video", "16384", "16384", 24, 24, 128, False, 2048, 2048, 77, fused=True),
        # a pair of images (with and without guidance) at a UNet level of width 640: few tokens, a shared prompt
        _prefix("prefix_pair_small", 77, "64,64", "64,64", 10, 10, 64, False),
        # one new token for each of 64 sequences that began with the same 8 k tokens
        _prefix("prefix_one_token", 8192, ",".join(["1"] * 64),
                ",".join(str(1 + (i * 211) % 509) for i in range(64)), 32, 8, 128, True, lse=True),
        # ragged continuations of one context, causal, shared key heads
        _prefix("prefix_continuations", 4001, "1,300,17,128,64,251,33,200,5,77", "1,300,17,128,64,251,33,200,5,77",
                32, 8, 128, True, lse=True),
        # four images that all attend to one reference image's tokens
        _prefix("prefix_reference_image", 4608, "1024,1024,1024,1024", "1024,1024,1024,1024", 24, 24, 128, False),
    ]


def _spread(rng, lo, hi):
    """A whole number whose logarithm is uniform over the range."""
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 1)))))))


def _text(lengths):
    return ",".join(map(str, lengths))


def draw(rng):
    op = rng.choice(("rope", "window", "window", "prefix", "prefix"))
    d = rng.choice((64, 72, 80, 96, 128))
    hkv = rng.choice((1, 2, 4, 8, 10))
    group = rng.choice((1, 1, 2, 3, 4, 8))
    if op == "rope":
        rows = [_spread(rng, 1, 3000) for _ in range(_spread(rng, 1, 12))]
        rot = rng.choice((d, d, 8 * (d // 16), 8))
        c = _rope(None, _text(rows), hkv * group, hkv, d, rot, rng.choice(("neighbours", "halves")),
                  rng.choice(("rms", "rms", "layer", "none")), rng.random() < 0.3, max(rows) + _spread(rng, 1, 50000),
                  rng.random() < 0.5, rng.random() < 0.5)
    elif op == "window":
        one = rng.random() < 0.35
        batch = _spread(rng, 1, 24)
        if one:
            q = [rng.choice((1, 1, 1, 2, 5)) for _ in range(batch)]
            k = [_spread(rng, 5, 12000) for _ in q]
        else:
            q = k = [_spread(rng, 1, min(8192, 16384 // batch)) for _ in range(batch)]
        # the padded scores of the plain form stay below the longest listed sequence's
        while batch * max(q) * max(k) * hkv * group > 16384 * 16384 * 12 and group > 1:
            group -= 1
        while batch * max(q) * max(k) * hkv * group > 16384 * 16384 * 12 and hkv > 1:
            hkv //= 2
        causal = one or rng.random() < 0.6
        c = _window(None, _text(q), _text(k), hkv * group, hkv, d, causal, _spread(rng, 8, 4096),
                    0 if causal else rng.choice((-1, 0, _spread(rng, 8, 2048))), rng.choice((0, 1, 4, _spread(rng, 2, 300))),
                    rng.random() < 0.3, not one and rng.random() < 0.5)
    else:
        one = rng.random() < 0.5
        batch = _spread(rng, 2, 64 if one else 12)
        if one:
            q = [rng.choice((1, 1, 1, 2, 3)) for _ in range(batch)]
            k = [n + _spread(rng, 1, 1000) - 1 for n in q]
        else:
            q = k = [_spread(rng, 1, min(2000, 8192 // batch)) for _ in range(batch)]
        prefix = _spread(rng, 16, 12000)
        while batch * max(q) * (prefix + max(k)) * hkv * group > 16384 * 16384 * 4 and group > 1:
            group -= 1
        while batch * max(q) * (prefix + max(k)) * hkv * group > 16384 * 16384 * 4 and hkv > 1:
            hkv //= 2
        c = _prefix(None, prefix, _text(q), _text(k), hkv * group, hkv, d, one or rng.random() < 0.6, rng.random() < 0.3)
    del c["name"]
    return c


# ------------------------------------------------------------------ inputs
def _lengths(text):
    return [int(v) for v in text.split(",")]


def _offsets(lengths):
    cu = [0]
    for n in lengths:
        cu.append(cu[-1] + n)
    return cu


def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)

    def normal(*shape, std=1.0, dtype=torch.bfloat16):
        return (torch.randn(*shape, generator=g, device="cuda") * std).to(dtype)

    def offsets(lengths):
        return torch.tensor(_offsets(lengths), dtype=torch.int32, device="cuda")

    s = dict(case)
    d, hq = case["d"], case["hq"]
    if case["op"] == "rope":
        rows, hk, rot = _lengths(case["rows"]), case["hk"], case["rot"]
        total = sum(rows)
        # a projection's output: heads of different size, some channels larger than the rest
        size = torch.exp(0.5 * torch.randn(hq + 2 * hk, d, generator=g, device="cuda"))
        qkv = (torch.randn(total, hq + 2 * hk, d, generator=g, device="cuda") * size).to(torch.bfloat16)
        s["Q"], s["K"] = qkv[:, :hq], qkv[:, hq:hq + hk]
        if not case["fused"]:
            s["Q"], s["K"] = s["Q"].contiguous(), s["K"].contiguous()
        s["cu"] = offsets(rows) if len(rows) > 1 else None
        # a model's table of cosines and sines, angle = position / 10000^(2 i / rot)
        rate = torch.pow(10000.0, -torch.arange(0, rot, 2, dtype=torch.float64, device="cuda") / rot)
        angle = torch.arange(case["table"], dtype=torch.float64, device="cuda")[:, None] * rate
        s["cos"], s["sin"] = angle.cos().float(), angle.sin().float()
        s["positions"] = (torch.randint(case["table"], (total,), generator=g, device="cuda", dtype=torch.int32)
                          if case["given"] else None)
        normed = case["norm"] != "none"
        s["wq"], s["wk"] = ((1 + normal(d, std=0.2, dtype=torch.float32)).to(torch.bfloat16) if normed else None
                            for _ in range(2))
        s["bq"], s["bk"] = (normal(d, std=0.1) if case["bias"] else None for _ in range(2))
        s["eps"] = 1e-6
        s["Q_out"] = torch.empty(total, hq, d, dtype=torch.bfloat16, device="cuda")
        s["K_out"] = torch.empty(total, hk, d, dtype=torch.bfloat16, device="cuda")
        return s
    lq, lk, hkv = _lengths(case["q"]), _lengths(case["k"]), case["hkv"]
    total_q, total_k = sum(lq), sum(lk)
    # normalised queries and keys with a gain: scores of standard deviation about 2
    if case.get("fused"):
        qkv = normal(total_q, (hq + 2 * hkv) * d, std=1.4).view(total_q, hq + 2 * hkv, d)
        s["Q"], s["K"], s["V"] = qkv[:, :hq], qkv[:, hq:hq + hkv], qkv[:, hq + hkv:]
    else:
        s["Q"], s["K"] = normal(total_q, hq, d, std=1.4), normal(total_k, hkv, d, std=1.4)
        s["V"] = normal(total_k, hkv, d)
    if case["op"] == "prefix":
        s["prefix_K"], s["prefix_V"] = normal(case["prefix"], hkv, d, std=1.4), normal(case["prefix"], hkv, d)
    s["cu_q"], s["cu_k"] = offsets(lq), offsets(lk)
    s["max_q"], s["max_k"] = max(lq), max(lk)
    s["scale"] = 1.0 / math.sqrt(d)
    s["O"] = torch.empty(total_q, hq, d, dtype=torch.bfloat16, device="cuda")
    s["LSE"] = torch.empty(hq, total_q, dtype=torch.float32, device="cuda") if case["lse"] else None
    s["workspace"] = torch.empty(WORKSPACE, dtype=torch.uint8, device="cuda")
    return s


# ------------------------------------------------------------------ the plain form
def _plain_rope_one(v, w, b, s, cos, sin):
    """The norm of each head's channels, then the rotation of pairs of them."""
    v = v.float()
    if s["norm"] != "none":
        if s["norm"] == "layer":
            v = v - v.mean(dim=-1, keepdim=True)
        v = v * torch.rsqrt(v.square().mean(dim=-1, keepdim=True) + s["eps"])
    if w is not None:
        v = v * w.float()
    if b is not None:
        v = v + b.float()
    rot = s["rot"]
    turned, rest = v[..., :rot], v[..., rot:]
    if s["pairs"] == "halves":
        x, y = turned[..., :rot // 2], turned[..., rot // 2:]
        turned = torch.cat([x * cos - y * sin, y * cos + x * sin], dim=-1)
    else:
        x, y = turned[..., 0::2], turned[..., 1::2]
        turned = torch.stack([x * cos - y * sin, y * cos + x * sin], dim=-1).flatten(-2)
    return torch.cat([turned, rest], dim=-1).to(torch.bfloat16)


def _plain_rope(s):
    if s["positions"] is not None:
        at = s["positions"].long()
    else:
        at = torch.arange(s["Q"].shape[0], device=s["Q"].device)
        if s["cu"] is not None:
            cu = s["cu"].long()
            at = at - cu[torch.searchsorted(cu, at, right=True) - 1]
    cos, sin = s["cos"][at][:, None], s["sin"][at][:, None]
    return (_plain_rope_one(s["Q"], s["wq"], s["bq"], s, cos, sin), _plain_rope_one(s["K"], s["wk"], s["bk"], s, cos, sin))


def _plain_attention(s):
    """Softmax attention over the sequences padded to the longest, masked, in 32 bits; a shared prefix's
    scores come from one product with all queries."""
    Q, K, V, cuq, cuk = s["Q"].float(), s["K"].float(), s["V"].float(), s["cu_q"].long(), s["cu_k"].long()
    hq, hkv, d, mq, mk = s["hq"], s["hkv"], s["d"], s["max_q"], s["max_k"]
    group = hq // hkv
    lq, lk = cuq[1:] - cuq[:-1], cuk[1:] - cuk[:-1]
    batch = lq.numel()
    iq = torch.arange(mq, device=Q.device)
    ik = torch.arange(mk, device=Q.device)
    at_q = torch.minimum(cuq[:-1, None] + iq, cuq[-1] - 1)
    at_k = torch.clamp(torch.minimum(cuk[:-1, None] + ik, cuk[-1] - 1), min=0)
    q = Q[at_q].transpose(1, 2).contiguous()                                   # [batch, hq, mq, d]
    k = K[at_k].repeat_interleave(group, dim=2).permute(0, 2, 3, 1).contiguous()
    v = V[at_k].repeat_interleave(group, dim=2).transpose(1, 2).contiguous()
    scores = torch.matmul(q, k).mul_(s["scale"])                               # [batch, hq, mq, mk]
    place = iq[None, :, None] + (lk - lq)[:, None, None]                       # the query's own key
    seen = (ik < lk[:, None])[:, None, :].expand(batch, mq, mk)
    if s["causal"]:
        seen = seen & (ik <= place)
    if s["op"] == "window":
        inside = torch.ones_like(seen)
        if s["left"] >= 0:
            inside = inside & (ik >= place - s["left"])
        if s["right"] >= 0:
            inside = inside & (ik <= place + s["right"])
        seen = seen & (inside | (ik < s["sinks"]))
    scores.masked_fill_(~seen[:, None], -math.inf)
    top = scores.amax(dim=-1, keepdim=True)
    if s["op"] == "prefix":
        pk = s["prefix_K"].float().repeat_interleave(group, dim=1).permute(1, 2, 0).contiguous()
        pv = s["prefix_V"].float().repeat_interleave(group, dim=1).transpose(0, 1).contiguous()
        rows = q.transpose(0, 1).reshape(hq, batch * mq, d)
        first = torch.matmul(rows, pk).mul_(s["scale"])                        # [hq, batch mq, prefix]
        top = torch.maximum(top, first.amax(dim=-1).view(hq, batch, mq).transpose(0, 1)[..., None])
    top = torch.where(top == -math.inf, torch.zeros_like(top), top)
    p = scores.sub_(top).exp_()
    total = p.sum(dim=-1, keepdim=True)
    out = torch.matmul(p, v)
    if s["op"] == "prefix":
        p = first.sub_(top.transpose(0, 1).reshape(hq, batch * mq, 1)).exp_()
        total = total + p.sum(dim=-1).view(hq, batch, mq).transpose(0, 1)[..., None]
        out = out + torch.matmul(p, pv).view(hq, batch, mq, d).transpose(0, 1)
    out = torch.where(total > 0, out / total, torch.zeros_like(out))
    row = torch.arange(Q.shape[0], device=Q.device)
    b = torch.searchsorted(cuq, row, right=True) - 1
    O = out[b, :, row - cuq[b]].to(torch.bfloat16)
    if s["LSE"] is None:
        return O
    return O, (top + total.log()).squeeze(-1)[b, :, row - cuq[b]].t().contiguous()


# ------------------------------------------------------------------ the library's calls
def _own(s):
    import bit_diffusion_model_svdq_amd as S
    if s["op"] == "rope":
        kinds = {"none": S.SVDQ_NORM_NONE, "rms": S.SVDQ_NORM_RMS, "layer": S.SVDQ_NORM_LAYER}
        pairs = {"neighbours": S.SVDQ_ROPE_NEIGHBOURS, "halves": S.SVDQ_ROPE_HALVES}
        S.svdq_qk_norm_rope_forward(s["Q"], s["K"], s["cu"], s["positions"], kinds[s["norm"]], s["wq"], s["bq"], s["wk"],
                                    s["bk"], s["eps"], s["cos"], s["sin"], pairs[s["pairs"]], s["Q_out"], s["K_out"])
        return s["Q_out"], s["K_out"]
    if s["op"] == "window":
        S.svdq_attention_window_forward(s["Q"], s["K"], s["V"], s["cu_q"], s["cu_k"], s["scale"], s["causal"], s["left"],
                                        s["right"], s["sinks"], s["O"], s["LSE"], s["workspace"])
    else:
        S.svdq_attention_prefix_forward(s["Q"], s["prefix_K"], s["prefix_V"], s["K"], s["V"], s["cu_q"], s["cu_k"],
                                        s["scale"], s["causal"], s["O"], s["LSE"], s["workspace"])
    return s["O"] if s["LSE"] is None else (s["O"], s["LSE"])


def run(state):
    if own:
        return _own(state)
    return _plain_rope(state) if state["op"] == "rope" else _plain_attention(state)


# ------------------------------------------------------------------ work and the 64-bit values
def _visible(case, nq, nk):
    """For every query of a sequence: (first key of its window, one past its last, first keys that it
    sees in any case)."""
    p = np.arange(nq, dtype=np.int64) + nk - nq
    lo, hi, sinks = np.zeros(nq, np.int64), np.full(nq, nk, np.int64), np.zeros(nq, np.int64)
    if case["op"] == "window":
        if case["left"] >= 0:
            lo = np.clip(p - case["left"], 0, nk)
        if case["right"] >= 0:
            hi = np.clip(p + case["right"] + 1, 0, nk)
        sinks = np.full(nq, min(case["sinks"], nk))
    if case["causal"]:
        hi, sinks = np.minimum(hi, np.clip(p + 1, 0, nk)), np.minimum(sinks, np.clip(p + 1, 0, nk))
    return lo, np.maximum(hi, lo), sinks


def work(case):
    if case["op"] == "rope":
        n = sum(_lengths(case["rows"])) * (case["hq"] + case["hk"]) * case["d"]
        used = sum(_lengths(case["rows"])) if case["given"] else max(_lengths(case["rows"]))
        return {"bytes": 4 * n + 4 * case["rot"] * min(used, case["table"]), "flops": 8 * n}
    pairs = keys = 0
    for nq, nk in zip(_lengths(case["q"]), _lengths(case["k"])):
        lo, hi, sinks = _visible(case, nq, nk)
        pairs += int((hi - lo + np.minimum(sinks, lo) + np.maximum(sinks - hi, 0)).sum())
        first = int(sinks.max(initial=0))
        begin = max(int(lo.min(initial=nk)), first)
        keys += first + max(int(hi.max(initial=0)) - begin, 0)
        if case["op"] == "prefix":
            pairs += nq * case["prefix"]
    if case["op"] == "prefix":
        keys += case["prefix"]
    queries = sum(_lengths(case["q"])) * case["hq"]
    return {"bytes": 4 * queries * case["d"] + 4 * keys * case["hkv"] * case["d"] + (4 * queries if case["lse"] else 0),
            "flops": 4 * pairs * case["hq"] * case["d"]}


def _exact_rope(s):
    rows, rot = _lengths(s["rows"]), s["rot"]
    at = torch.cat([torch.arange(n) for n in rows]).cuda() if s["positions"] is None else s["positions"].long()
    z = torch.complex(s["cos"].double()[at], s["sin"].double()[at])[:, None]   # a pair is turned by z
    out = []
    for v, w, b in ((s["Q"], s["wq"], s["bq"]), (s["K"], s["wk"], s["bk"])):
        v = v.double()
        if s["norm"] != "none":
            mean = v.mean(-1, keepdim=True) if s["norm"] == "layer" else 0.0
            v = (v - mean) / torch.sqrt(((v - mean) ** 2).mean(-1, keepdim=True) + s["eps"])
        v = v * (w.double() if w is not None else 1.0) + (b.double() if b is not None else 0.0)
        a = v.clone()
        first, second = (slice(0, rot // 2), slice(rot // 2, rot)) if s["pairs"] == "halves" else (slice(0, rot, 2), slice(1, rot, 2))
        t = torch.complex(v[..., first].contiguous(), v[..., second].contiguous()) * z
        a[..., first], a[..., second] = t.real, t.imag
        out.append(a)
    return tuple(out)


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "rope":
        return _exact_rope(s)
    group, d = case["hq"] // case["hkv"], case["d"]
    O = torch.zeros(s["Q"].shape, dtype=torch.float64, device="cuda")
    lse = torch.full((case["hq"], O.shape[0]), -math.inf, dtype=torch.float64, device="cuda")
    q0 = k0 = 0
    for nq, nk in zip(_lengths(case["q"]), _lengths(case["k"])):
        lo, hi, sinks = (torch.from_numpy(x).cuda()[:, None] for x in _visible(case, nq, nk))
        j = torch.arange(nk, device="cuda")
        hidden = ~(((j >= lo) & (j < hi)) | (j < sinks))
        for h in range(case["hq"]):
            k = s["K"][k0:k0 + nk, h // group].double()
            v = s["V"][k0:k0 + nk, h // group].double()
            a = ((s["Q"][q0:q0 + nq, h].double() @ k.t()) / math.sqrt(d)).masked_fill(hidden, -math.inf)
            if case["op"] == "prefix":
                a = torch.cat([s["Q"][q0:q0 + nq, h].double() @ s["prefix_K"][:, h // group].double().t() / math.sqrt(d), a], 1)
                v = torch.cat([s["prefix_V"][:, h // group].double(), v])
            some = a.amax(1) > -math.inf
            O[q0:q0 + nq, h] = torch.where(some[:, None], torch.nan_to_num(torch.softmax(a, dim=1)) @ v, 0.0)
            lse[h, q0:q0 + nq] = torch.logsumexp(a, dim=1)
        q0, k0 = q0 + nq, k0 + nk
    return (O, lse) if case["lse"] else O
