"""What is measured of the block operators around the quantized linears: attention over packed
sequences, the norms around a block with its gate and residual, and the 16-bit linear.

`run` computes them in their plain form (elementary torch operations in 32 bits, rounded once),
or, where `own` is true, through the library's entry points.  Inputs are bf16 unless a case says
otherwise; packed batches carry their row offsets `cu` [batch + 1] on the GPU, as the calls take
them.
"""
import math

import torch

own = False

# A serving program keeps one workspace for all its layers; 64 MiB is also what the library's
# allocation-free forward holds.
WORKSPACE = 64 << 20


# ------------------------------------------------------------------ cases
def _attention(name, q, k, hq, hkv, d, causal, lse=False, fused=False):
    """q, k: the lengths of the sequences, comma separated; fused: Q, K and V are column slices of
    one [tokens, (hq + 2 hkv) d] projection output."""
    return dict(name=name, op="attention", q=q, k=k, hq=hq, hkv=hkv, d=d, causal=causal, lse=lse, fused=fused)


def _norm(name, rows, width, post, pre, fp32, affine):
    """rows: the lengths of the sequences; fp32: the residual stream's type (else bf16)."""
    return dict(name=name, op="norm", rows=rows, width=width, post=post, pre=pre, fp32=fp32, affine=affine)


def _linear(name, m, k, n, act, residual, fp32):
    return dict(name=name, op="linear", m=m, k=k, n=n, act=act, residual=residual, fp32=fp32)


def listed():
    return [
        # a text encoder on one prompt of 77 tokens, width 640: latency is all there is
        _attention("attention_prompt_77", "77", "77", 10, 10, 64, True, fused=True),
        # one new token for each of 16 sequences against long, unequal histories, shared key heads;
        # the log-sum-exp comes along, as a program needs it that joins partial results
        _attention("attention_one_token", ",".join(["1"] * 16),
                   "8192,517,4096,1,2049,7777,63,3000,6143,129,1024,5000,2500,8000,64,900", 32, 8, 128, True,
                   lse=True),
        # prompts of different lengths packed behind each other, causal, shared key heads
        _attention("attention_packed_prompts", "1,17,511,2048,1023,4096,333,64", "1,17,511,2048,1023,4096,333,64",
                   32, 8, 128, True, lse=True),
        # a UNet level of width 640: two images' tokens against their prompts' keys
        _attention("attention_cross_77", "4096,4096", "77,77", 10, 10, 64, False),
        # the joint attention of a DiT block (4608 tokens of width 3072), read out of the fused
        # QKV projection's output
        _attention("attention_dit_block", "4608", "4608", 24, 24, 128, False, fused=True),
        # the same block on a large image: the longest sequence
        _attention("attention_large_image", "16384", "16384", 24, 24, 128, False, fused=True),
        # the prompt's rows beside an image: latency
        _norm("norm_prompt_154", "77,77", 640, "none", "layer", False, False),
        # between a DiT block's linears: gate, residual, LayerNorm and its modulation
        _norm("norm_dit_block", "4608", 3072, "none", "layer", False, False),
        # RMS norms before and after the block over a 32-bit residual stream, three images
        _norm("norm_sandwich_fp32", "16384,9001,4099", 1280, "rms", "rms", True, True),
        # the six modulation vectors of a DiT block from two conditioning vectors: the weight's bytes
        _linear("linear_modulation", 2, 3072, 18432, "none", False, False),
        # a ragged batch through a 16-bit output projection onto a 32-bit residual stream
        _linear("linear_residual_odd", 1155, 1288, 1290, "none", True, True),
        # a block's up projection kept in 16 bits, GELU in its epilogue
        _linear("linear_mlp_up", 4608, 3072, 12288, "gelu", False, False),
    ]


def _spread(rng, lo, hi):
    """A whole number whose logarithm is uniform over the range."""
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 1)))))))


def draw(rng):
    op = rng.choice(("attention", "attention", "norm", "linear"))
    if op == "attention":
        kind = rng.choice(("self", "self", "one", "cross"))
        batch = _spread(rng, 1, 24)
        d = rng.choice((64, 80, 96, 128))
        hkv = rng.choice((1, 2, 4, 8, 10))
        group = rng.choice((1, 1, 2, 3, 4, 8))
        if kind == "one":
            q = [rng.choice((1, 1, 1, 2, 5)) for _ in range(batch)]
            k = [_spread(rng, 5, 12000) for _ in q]
        elif kind == "cross":
            q = [_spread(rng, 16, 4096) for _ in range(batch)]
            k = [_spread(rng, 1, 500) for _ in q]
        else:
            most = min(8192, 16384 // batch)
            q = [_spread(rng, 1, most) for _ in range(batch)]
            k = q
        # the padded scores of the plain form stay below the longest listed sequence's
        while batch * max(q) * max(k) * hkv * group > 16384 * 16384 * 12 and group > 1:
            group -= 1
        while batch * max(q) * max(k) * hkv * group > 16384 * 16384 * 12 and hkv > 1:
            hkv //= 2
        c = _attention(None, ",".join(map(str, q)), ",".join(map(str, k)), hkv * group, hkv, d,
                       kind != "cross" and rng.random() < 0.6, rng.random() < 0.3, kind == "self" and rng.random() < 0.5)
    elif op == "norm":
        rows = [_spread(rng, 1, 8000) for _ in range(_spread(rng, 1, 8))]
        c = _norm(None, ",".join(map(str, rows)), 8 * _spread(rng, 16, 512), rng.choice(("none", "rms", "layer")),
                  rng.choice(("layer", "rms")), rng.random() < 0.3, rng.random() < 0.5)
    else:
        m, k, n = _spread(rng, 1, 8192), 8 * _spread(rng, 8, 768), _spread(rng, 16, 12288)
        while m * k * n > 4608 * 3072 * 12288:
            m //= 2
        c = _linear(None, m, k, n, rng.choice(("none", "gelu", "silu")), rng.random() < 0.5, rng.random() < 0.3)
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

    def outliers(width, share=0.005, factor=20.0):
        """Channel factors: a few input channels of a diffusion model are far larger than the rest."""
        f = torch.ones(width, device="cuda")
        f[torch.rand(width, generator=g, device="cuda") < share] = factor
        return f

    s = dict(case)
    if case["op"] == "attention":
        lq, lk = _lengths(case["q"]), _lengths(case["k"])
        hq, hkv, d = case["hq"], case["hkv"], case["d"]
        cuq, cuk = _offsets(lq), _offsets(lk)
        # normalised queries and keys with a gain: scores of standard deviation about 2
        if case["fused"]:
            qkv = normal(cuq[-1], (hq + 2 * hkv) * d, std=1.4).view(cuq[-1], hq + 2 * hkv, d)
            s["Q"], s["K"], s["V"] = qkv[:, :hq], qkv[:, hq:hq + hkv], qkv[:, hq + hkv:]
        else:
            s["Q"], s["K"] = normal(cuq[-1], hq, d, std=1.4), normal(cuk[-1], hkv, d, std=1.4)
            s["V"] = normal(cuk[-1], hkv, d)
        s["cu_q"] = torch.tensor(cuq, dtype=torch.int32, device="cuda")
        s["cu_k"] = torch.tensor(cuk, dtype=torch.int32, device="cuda")
        s["max_q"], s["max_k"] = max(lq), max(lk)
        s["scale"] = 1.0 / math.sqrt(d)
        s["O"] = torch.empty(cuq[-1], hq, d, dtype=torch.bfloat16, device="cuda")
        s["LSE"] = torch.empty(hq, cuq[-1], dtype=torch.float32, device="cuda") if case["lse"] else None
        s["workspace"] = torch.empty(WORKSPACE, dtype=torch.uint8, device="cuda")
    elif case["op"] == "norm":
        rows = _lengths(case["rows"])
        cu, width, batch = _offsets(rows), case["width"], len(rows)
        dt = torch.float32 if case["fp32"] else torch.bfloat16
        s["cu"] = torch.tensor(cu, dtype=torch.int32, device="cuda")
        s["x"] = (torch.randn(cu[-1], width, generator=g, device="cuda") * outliers(width)).to(dt)
        s["y"] = normal(cu[-1], width, std=0.7)
        # gate, scale and shift are column slices of the block's modulation vectors
        mod = normal(batch, 6 * width, std=0.3)
        s["shift"], s["scale"], s["gate"] = mod[:, :width], mod[:, width:2 * width], mod[:, 2 * width:3 * width]
        s["w_post"] = (1 + normal(width, std=0.1, dtype=torch.float32)).to(torch.bfloat16)
        s["w_pre"] = (1 + normal(width, std=0.1, dtype=torch.float32)).to(torch.bfloat16) if case["affine"] else None
        s["b_pre"] = normal(width, std=0.1) if case["affine"] and case["pre"] == "layer" else None
        s["residual_scale"], s["branch_scale"], s["eps"] = 1.0, 0.5 if case["post"] == "rms" else 1.0, 1e-6
        s["x_out"] = torch.empty_like(s["x"])
        s["h"] = torch.empty(cu[-1], width, dtype=torch.bfloat16, device="cuda")
    else:
        m, k, n = case["m"], case["k"], case["n"]
        dt = torch.float32 if case["fp32"] else torch.bfloat16
        s["X"] = (torch.randn(m, k, generator=g, device="cuda") * outliers(k)).to(torch.bfloat16)
        s["W"] = normal(n, k, std=1.0 / math.sqrt(k))
        s["bias"] = normal(n, std=0.1)
        s["residual"] = normal(m, n, dtype=dt) if case["residual"] else None
        s["Y"] = torch.empty(m, n, dtype=dt, device="cuda")
        s["workspace"] = torch.empty(WORKSPACE, dtype=torch.uint8, device="cuda")
    return s


# ------------------------------------------------------------------ the plain form
def _plain_attention(s):
    """Softmax attention over the sequences padded to the longest, masked, in 32 bits."""
    Q, K, V, cuq, cuk = s["Q"].float(), s["K"].float(), s["V"].float(), s["cu_q"].long(), s["cu_k"].long()
    hq, hkv, d = s["hq"], s["hkv"], s["d"]
    lq, lk = cuq[1:] - cuq[:-1], cuk[1:] - cuk[:-1]
    batch = lq.numel()
    pq = torch.arange(s["max_q"], device=Q.device)
    pk = torch.arange(s["max_k"], device=Q.device)
    q = Q[torch.minimum(cuq[:-1, None] + pq, cuq[-1] - 1)]                    # [batch, max_q, hq, d]
    at = torch.clamp(torch.minimum(cuk[:-1, None] + pk, cuk[-1] - 1), min=0)
    k = K[at].repeat_interleave(hq // hkv, dim=2)
    v = V[at].repeat_interleave(hq // hkv, dim=2)
    q = q.transpose(1, 2).reshape(batch * hq, s["max_q"], d)
    k = k.permute(0, 2, 3, 1).reshape(batch * hq, d, s["max_k"]).contiguous()
    v = v.transpose(1, 2).reshape(batch * hq, s["max_k"], d).contiguous()
    scores = torch.bmm(q, k).mul_(s["scale"]).view(batch, hq, s["max_q"], s["max_k"])
    seen = (pk < lk[:, None])[:, None, None, :]
    if s["causal"]:   # the last query sees the last key
        seen = seen & (pk <= (pq[None, :, None] + (lk - lq)[:, None, None]))[:, None]
    scores.masked_fill_(~seen, -math.inf)
    top = scores.amax(dim=-1, keepdim=True)
    top = torch.where(top == -math.inf, torch.zeros_like(top), top)
    p = scores.sub_(top).exp_()
    total = p.sum(dim=-1, keepdim=True)
    out = torch.bmm(p.view(batch * hq, s["max_q"], s["max_k"]), v).view(batch, hq, s["max_q"], d)
    out = torch.where(total > 0, out / total, torch.zeros_like(out))
    row = torch.arange(Q.shape[0], device=Q.device)
    b = torch.searchsorted(cuq, row, right=True) - 1
    O = out[b, :, row - cuq[b]].to(torch.bfloat16)
    if s["LSE"] is None:
        return O
    return O, (top + total.log()).squeeze(-1)[b, :, row - cuq[b]].t().contiguous()


def _plain_normalise(v, kind, eps):
    if kind == "none":
        return v
    if kind == "layer":
        v = v - v.mean(dim=-1, keepdim=True)
    return v * torch.rsqrt(v.square().mean(dim=-1, keepdim=True) + eps)


def _plain_norm(s):
    """x' = a x + c gate post(y), h = pre(x') (1 + scale) + shift, in 32 bits."""
    row = torch.arange(s["x"].shape[0], device=s["x"].device)
    b = torch.searchsorted(s["cu"].long(), row, right=True) - 1
    u = _plain_normalise(s["y"].float(), s["post"], s["eps"])
    if s["post"] != "none":
        u = u * s["w_post"].float()
    x = s["residual_scale"] * s["x"].float() + s["branch_scale"] * s["gate"].float()[b] * u
    h = _plain_normalise(x, s["pre"], s["eps"])
    if s["w_pre"] is not None:
        h = h * s["w_pre"].float()
    if s["b_pre"] is not None:
        h = h + s["b_pre"].float()
    h = h * (1 + s["scale"].float()[b]) + s["shift"].float()[b]
    return x.to(s["x"].dtype), h.to(torch.bfloat16)


def _plain_linear(s):
    """act(X W^T + bias) + residual, in 32 bits."""
    y = s["X"].float() @ s["W"].float().t() + s["bias"].float()
    if s["act"] == "gelu":
        y = 0.5 * y * (1 + torch.tanh(math.sqrt(2 / math.pi) * (y + 0.044715 * y * y * y)))
    elif s["act"] == "silu":
        y = y / (1 + torch.exp(-y))
    if s["residual"] is not None:
        y = y + s["residual"].float()
    return y.to(s["Y"].dtype)


# ------------------------------------------------------------------ the library's calls
def _own(s):
    import bit_diffusion_model_svdq_amd as S
    if s["op"] == "attention":
        S.svdq_attention_forward(s["Q"], s["K"], s["V"], s["cu_q"], s["cu_k"], s["scale"], s["causal"], s["O"],
                                 s["LSE"], s["workspace"])
        return s["O"] if s["LSE"] is None else (s["O"], s["LSE"])
    if s["op"] == "norm":
        kinds = {"none": S.SVDQ_NORM_NONE, "rms": S.SVDQ_NORM_RMS, "layer": S.SVDQ_NORM_LAYER}
        S.svdq_block_norm_forward(s["x"], s["y"], s["cu"], kinds[s["post"]],
                                  s["w_post"] if s["post"] != "none" else None, s["gate"], s["residual_scale"],
                                  s["branch_scale"], kinds[s["pre"]], s["w_pre"], s["b_pre"], s["scale"], s["shift"],
                                  s["eps"], s["x_out"], s["h"])
        return s["x_out"], s["h"]
    acts = {"none": S.SVDQ_ACT_NONE, "gelu": S.SVDQ_ACT_GELU_TANH, "silu": S.SVDQ_ACT_SILU}
    S.svdq_linear_bf16_forward(s["X"], s["W"], s["bias"], acts[s["act"]], s["residual"], s["Y"], s["workspace"])
    return s["Y"]


def run(state):
    if own:
        return _own(state)
    return {"attention": _plain_attention, "norm": _plain_norm, "linear": _plain_linear}[state["op"]](state)


# ------------------------------------------------------------------ work and the 64-bit values
def work(case):
    if case["op"] == "attention":
        lq, lk = _lengths(case["q"]), _lengths(case["k"])
        pairs = 0
        for q, k in zip(lq, lk):
            if case["causal"]:   # query i of q sees max(0, i + 1 + k - q) keys
                first = max(0, q - k)
                pairs += sum((first + 1 + k - q, k)) * (q - first) // 2 if q > first else 0
            else:
                pairs += q * k
        rows = 2 * sum(lq) * case["hq"] * case["d"] + 2 * sum(lk) * case["hkv"] * case["d"]
        return {"bytes": 2 * rows + (4 * sum(lq) * case["hq"] if case["lse"] else 0),
                "flops": 4 * pairs * case["hq"] * case["d"]}
    if case["op"] == "norm":
        n = sum(_lengths(case["rows"])) * case["width"]
        return {"bytes": n * (2 * (4 if case["fp32"] else 2) + 4), "flops": 12 * n}
    m, k, n = case["m"], case["k"], case["n"]
    out = 4 if case["fp32"] else 2
    return {"bytes": 2 * (m * k + n * k + n) + m * n * out * (2 if case["residual"] else 1), "flops": 2 * m * k * n}


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "attention":
        group = case["hq"] // case["hkv"]
        O = torch.zeros(s["Q"].shape, dtype=torch.float64, device="cuda")
        lse = torch.full((case["hq"], O.shape[0]), -math.inf, dtype=torch.float64, device="cuda")
        q0 = k0 = 0
        for nq, nk in zip(_lengths(case["q"]), _lengths(case["k"])):
            for h in range(case["hq"]):
                q = s["Q"][q0:q0 + nq, h].double()
                k = s["K"][k0:k0 + nk, h // group].double()
                v = s["V"][k0:k0 + nk, h // group].double()
                a = (q @ k.t()) / math.sqrt(case["d"])
                if case["causal"]:
                    a = a.masked_fill(torch.ones_like(a, dtype=torch.bool).triu(nk - nq + 1), -math.inf)
                some = a.amax(1) > -math.inf
                O[q0:q0 + nq, h] = torch.where(some[:, None], torch.nan_to_num(torch.softmax(a, dim=1)) @ v, 0.0)
                lse[h, q0:q0 + nq] = torch.logsumexp(a, dim=1)
            q0, k0 = q0 + nq, k0 + nk
        return (O, lse) if case["lse"] else O
    if case["op"] == "norm":
        xs, hs, r0 = [], [], 0

        def norm(t, kind):
            if kind == "none":
                return t
            mean = t.mean(1, keepdim=True) if kind == "layer" else 0.0
            return (t - mean) / torch.sqrt(((t - mean) ** 2).mean(1, keepdim=True) + s["eps"])

        for b, n in enumerate(_lengths(case["rows"])):
            y = norm(s["y"][r0:r0 + n].double(), case["post"])
            y = y * s["w_post"].double() if case["post"] != "none" else y
            x = s["x"][r0:r0 + n].double() * s["residual_scale"] + y * s["gate"][b].double() * s["branch_scale"]
            h = norm(x, case["pre"])
            h = h * s["w_pre"].double() if s["w_pre"] is not None else h
            h = h + s["b_pre"].double() if s["b_pre"] is not None else h
            xs.append(x)
            hs.append(h + h * s["scale"][b].double() + s["shift"][b].double())
            r0 += n
        return torch.cat(xs), torch.cat(hs)
    y = torch.nn.functional.linear(s["X"].double(), s["W"].double(), s["bias"].double())
    if case["act"] == "gelu":
        y = torch.nn.functional.gelu(y, approximate="tanh")
    elif case["act"] == "silu":
        y = y * torch.sigmoid(y)
    return y + s["residual"].double() if s["residual"] is not None else y
