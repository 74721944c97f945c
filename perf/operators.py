"""The operators of a mixture-of-experts layer around the load balancer, as cases to time and compare.

Four families: the gate (top-k expert IDs and weights from router logits, and its gradient), the
experts' grouped product in 8-bit floating point with a power-of-two scale for each block of 128
(forward, and a training step: output, input gradient in 8 bits too, weight gradient in bf16), the whole layer for a few tokens, and the AdamW
step over the experts' tensors with its states in 32 or in 8 bits.  Shapes follow the routing workloads
of this repository: expert matrices of (4096, 1536), (4096, 2048), (7168, 2048) and (5120, 1536), 128 to
384 experts, top-8, and the pairs that one expert-parallel rank receives.

`run` computes a case in plain torch operations in 32 bits, or, where `own` is set, by the package's
entry points; `exact` gives the definition's values in 64 bits.
"""
import math

import numpy as np
import torch
import torch.nn.functional as F

own = False

BLOCK = 128
MIX = (0x9E3779B9, 0x6A09E667, 0xBB67AE85)   # odd 32-bit fractions of the golden ratio, sqrt 2 and sqrt 3
BETA1, BETA2, EPS, DECAY, LR = 0.9, 0.95, 1e-8, 0.1, 3e-4


def listed():
    return [
        # one decode step of 64 sequences: group-limited routing with a selection bias, latency only
        dict(name="gate_decode", kind="gate", tokens=64, experts=256, k=8, groups=8, topk_groups=4, dtype="float32",
             bias=True, backward=False),
        # a training microbatch through the widest router, with the router's gradient; odd token count
        dict(name="gate_train", kind="gate", tokens=131071, experts=384, k=8, groups=1, topk_groups=1,
             dtype="bfloat16", bias=False, backward=True),
        # a handful of pairs over one rank's physical slots: the weights' bytes count
        dict(name="product_small", kind="product", pairs=40, groups=8, n=4096, k=1536, gather=1, train=False),
        # prefill, gate and up in one product: a rank's share of 8192 tokens x top-8, rows gathered by pair
        dict(name="product_prefill", kind="product", pairs=65536, groups=8, n=4096, k=4096, gather=8, train=False),
        # prefill, down: rows already in slot order, skewed groups with an empty one
        dict(name="product_ragged", kind="product", pairs=32749, groups=5, n=7168, k=2048, gather=0, train=False),
        # one training step of an expert matrix: output, input gradient, weight gradient
        dict(name="product_train", kind="product", pairs=16381, groups=3, n=2048, k=4096, gather=0, train=True),
        # decode of one sequence
        dict(name="layer_one", kind="layer", tokens=1, experts=128, k=8, hidden=4096, inter=1536, groups=1,
             topk_groups=1, weights="bfloat16", masked=False),
        # decode of a few sequences with 8-bit weights and group-limited routing
        dict(name="layer_eight_bit", kind="layer", tokens=7, experts=256, k=8, hidden=7168, inter=2048, groups=8,
             topk_groups=4, weights="float8", masked=False),
        # a full decode batch with padded rows: nearly every expert is hit
        dict(name="layer_batch", kind="layer", tokens=61, experts=160, k=8, hidden=5120, inter=1536, groups=1,
             topk_groups=1, weights="bfloat16", masked=True),
        # the small tensors of a layer (router, norms, biases): latency over many tensors
        dict(name="adamw_small", kind="adamw", tensors=12, size=5003, bits=32, grads="float32", copy=False),
        # one rank's native experts, states in 8 bits
        dict(name="adamw_eight_bit", kind="adamw", tensors=6, size=18874368, bits=8, grads="float32", copy=False),
        # the same with states in 32 bits, bf16 gradients and a bf16 copy of the weights for the forward pass
        dict(name="adamw_copy", kind="adamw", tensors=4, size=23592960, bits=32, grads="bfloat16", copy=True),
    ]


def _spread(rng, low, high):
    """A whole number of [low, high], even in its logarithm."""
    v = int(round(math.exp(rng.uniform(math.log(low), math.log(high)))))
    return max(low, min(high, v + 8 * (v in (384, 3072))))


def draw(rng):
    kind = rng.choice(("gate", "product", "product", "layer", "layer", "adamw"))
    if kind == "gate":
        groups, of = rng.choice(((1, 1), (1, 1), (8, 4), (4, 1), (5, 3)))
        experts = groups * max(-(-16 // groups), _spread(rng, 12, 384) // groups)
        return dict(kind=kind, tokens=_spread(rng, 1, 100000), experts=experts,
                    k=rng.randint(1, min(8, of * (experts // groups))), groups=groups, topk_groups=of,
                    dtype=rng.choice(("float32", "bfloat16")), bias=rng.random() < 0.5, backward=rng.random() < 0.5)
    if kind == "product":
        train = rng.random() < 0.4
        n, k = _spread(rng, 64, 4000 if train else 7168), _spread(rng, 64, 4096)
        return dict(kind=kind, pairs=min(_spread(rng, 1, 16000 if train else 65000), int(1e12 / (n * k))),
                    groups=rng.randint(1, 16), n=n, k=k, gather=0 if train else rng.choice((0, 1, 8)), train=train)
    if kind == "layer":
        groups, of = rng.choice(((1, 1), (1, 1), (4, 2)))
        experts = groups * max(4, _spread(rng, 8, 160) // groups)
        return dict(kind=kind, tokens=_spread(rng, 1, 64), experts=experts,
                    k=rng.randint(1, min(8, of * (experts // groups))), hidden=8 * _spread(rng, 32, 640),
                    inter=8 * _spread(rng, 16, 192), groups=groups, topk_groups=of,
                    weights=rng.choice(("bfloat16", "float8")), masked=rng.random() < 0.3)
    return dict(kind=kind, tensors=rng.randint(1, 12), size=_spread(rng, 1, 8000000), bits=rng.choice((32, 8)),
                grads=rng.choice(("float32", "bfloat16")), copy=rng.random() < 0.5)


# ------------------------------------------------------------------------------------------------ inputs

def _generator(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(int(seed) * 7919 + 13)
    return g


def _normal(g, *shape, dtype=torch.float32, std=1.0):
    return (torch.randn(shape, generator=g, device="cuda") * std).to(dtype)


def _padded(x, dim):
    """x with zeros up to a multiple of 128 along dim."""
    short = -x.shape[dim] % BLOCK
    return F.pad(x, [0, 0] * (x.dim() - 1 - dim % x.dim()) + [0, short]) if short else x


def _scale_code(amax):
    """The byte c of the smallest power of two 2**(c - 127) that brings amax to 448 at most."""
    bits = amax.float().view(torch.int32)
    code = (bits >> 23) - 8 + ((bits & 0x7FFFFF) > 0x600000).int()
    return code.clamp(1, 254).to(torch.uint8)


def _power(code):
    """2**(code - 127) as float32."""
    return (code.to(torch.int32) << 23).view(torch.float32)


def _blocks_quantised(w):
    """[G][N][K] in floats -> (8-bit [G][N][K up to 128], scale bytes [G][blocks of N][blocks of K])."""
    n = w.shape[1]
    p = _padded(_padded(w.float(), 2), 1)
    t = p.view(p.shape[0], p.shape[1] // BLOCK, BLOCK, p.shape[2] // BLOCK, BLOCK)
    code = _scale_code(t.abs().amax(dim=(2, 4)))
    q = (t * _power(254 - code)[:, :, None, :, None]).view(p.shape).to(torch.float8_e4m3fn)
    return q[:, :n].contiguous(), code.contiguous()


def _expert_weights(g, count, n, k, kind):
    if kind == "bfloat16":
        w = torch.empty((count, n, k), dtype=torch.bfloat16, device="cuda")
        for e in range(count):
            w[e] = torch.randn((n, k), generator=g, device="cuda") * k ** -0.5
        return w, None
    kp, blocks = -(-k // BLOCK) * BLOCK, -(-n // BLOCK)
    w = torch.empty((count, n, kp), dtype=torch.float8_e4m3fn, device="cuda")
    s = torch.empty((count, blocks, kp // BLOCK), dtype=torch.uint8, device="cuda")
    for e in range(count):
        q, c = _blocks_quantised(torch.randn((1, n, k), generator=g, device="cuda") * k ** -0.5)
        w[e], s[e] = q[0], c[0]
    return w, s


def _logits(g, tokens, experts, masked):
    """Router logits: noise, a skew over the experts, and (masked) experts switched off and padded tokens."""
    skew = torch.exp(0.7 * torch.randn(experts, generator=g, device="cuda"))
    x = 1.5 * torch.randn((tokens, experts), generator=g, device="cuda") + skew
    if masked:
        x[:, torch.rand(experts, generator=g, device="cuda") < 0.05] = -math.inf
        x[torch.rand(tokens, generator=g, device="cuda") < 0.1] = -math.inf
    return x


def _sizes(seed, pairs, groups):
    """Skewed group sizes that sum to `pairs`; with three groups or more one is empty."""
    r = np.random.default_rng(int(seed) * 31 + 5)
    p = r.dirichlet(np.full(groups, 1.5))
    if groups > 2:
        p[int(r.integers(groups))] = 0
    return r.multinomial(pairs, p / p.sum())


def prepare(case, seed):
    g, c = _generator(seed), case
    s = dict(case=dict(case))
    if c["kind"] == "gate":
        s["logits"] = _logits(g, c["tokens"], c["experts"], True).to(getattr(torch, c["dtype"]))
        s["bias"] = 0.3 * torch.randn(c["experts"], generator=g, device="cuda") if c["bias"] else None
        s["grad"] = _normal(g, c["tokens"], c["k"])
    elif c["kind"] == "product":
        sizes = _sizes(seed, c["pairs"], c["groups"])
        s["ends"] = [0] + [int(v) for v in np.cumsum(sizes)]
        s["offsets"] = torch.tensor(s["ends"], dtype=torch.int32, device="cuda")
        tokens = -(-c["pairs"] // c["gather"]) if c["gather"] else c["pairs"]
        # activations whose rows differ in size, with a few large channels
        spread = torch.exp(0.5 * torch.randn((tokens, 1), generator=g, device="cuda"))
        loud = 1 + 20 * (torch.rand(c["k"], generator=g, device="cuda") < 0.01).float()
        s["x"] = (torch.randn((tokens, c["k"]), generator=g, device="cuda") * spread * loud).to(torch.bfloat16)
        # which pair each slot-ordered row serves; its token is pair // top-k
        s["pairs"] = (torch.randperm(c["pairs"], generator=g, device="cuda").to(torch.int32)
                      if c["gather"] else None)
        w = torch.randn((c["groups"], c["n"], c["k"]), generator=g, device="cuda") * c["k"] ** -0.5
        s["w"], s["w_scale"] = _blocks_quantised(w)
        if c["train"]:
            s["wt"], s["wt_scale"] = _blocks_quantised(w.transpose(1, 2).contiguous())
            s["dy"] = _normal(g, c["pairs"], c["n"], dtype=torch.bfloat16, std=1e-3)
    elif c["kind"] == "layer":
        s["x"] = _normal(g, c["tokens"], c["hidden"], dtype=torch.bfloat16)
        s["logits"] = _logits(g, c["tokens"], c["experts"], c["masked"])
        s["bias"] = 0.3 * torch.randn(c["experts"], generator=g, device="cuda") if c["groups"] > 1 else None
        for name, n, k in (("gate", c["inter"], c["hidden"]), ("up", c["inter"], c["hidden"]),
                           ("down", c["hidden"], c["inter"])):
            s[name], s[name + "_scale"] = _expert_weights(g, c["experts"], n, k, c["weights"])
    else:
        sizes = [max(1, c["size"] - 61 * i) if c["size"] < 100000 or i == c["tensors"] - 1 else c["size"]
                 for i in range(c["tensors"])]
        s["params"] = [_normal(g, n, std=0.02) for n in sizes]
        s["grads"] = [_normal(g, n, dtype=getattr(torch, c["grads"]), std=1e-3) for n in sizes]
        s["step"], s["seed"] = 0, int(seed) & 0x7FFFFFFF
        s["copies"] = [torch.zeros(n, dtype=torch.bfloat16, device="cuda") for n in sizes] if c["copy"] else None
        if own:
            import moe_expert_load_layer_amd as ep
            s["opt"] = ep.AdamW(s["params"], bits=c["bits"], copies=s["copies"], beta1=BETA1, beta2=BETA2, eps=EPS,
                                weight_decay=DECAY, seed=s["seed"])
        elif c["bits"] == 32:
            s["m"], s["v"] = [torch.zeros_like(p) for p in s["params"]], [torch.zeros_like(p) for p in s["params"]]
        else:
            for name in ("m", "v"):
                s[name] = [torch.zeros(n, dtype=torch.uint8, device="cuda") for n in sizes]
                s[name + "_scale"] = [torch.ones(-(-n // BLOCK), dtype=torch.uint8, device="cuda") for n in sizes]
    return s


# ------------------------------------------------------------------------------------------------ plain forms

def _select(logits, bias, k, groups, topk_groups):
    """Top-k expert IDs (-1 where an expert is switched off) and softmax weights over the chosen logits."""
    l = logits.float()
    tokens, experts = l.shape
    score = l + bias if bias is not None else l
    if groups > 1:
        best = score.view(tokens, groups, -1).amax(dim=2)
        order = torch.sort(best, dim=1, descending=True, stable=True).indices[:, :topk_groups]
        kept = torch.zeros((tokens, groups), dtype=torch.bool, device=l.device).scatter_(1, order, True)
        score = score.masked_fill(~kept.repeat_interleave(experts // groups, dim=1), -math.inf)
    top = torch.sort(score, dim=1, descending=True, stable=True)
    chosen = top.values[:, :k] > -math.inf
    ids = torch.where(chosen, top.indices[:, :k], -1).to(torch.int32)
    z = l.gather(1, ids.clamp(min=0).long()).masked_fill(~chosen, -math.inf)
    e = torch.exp(z - z.amax(dim=1, keepdim=True).clamp(min=-3e38))
    e = torch.where(chosen, e, 0.0)
    total = e.sum(dim=1, keepdim=True)
    return ids, e / torch.where(total > 0, total, 1.0)


def _rows_quantised(x):
    """[M][K] -> values [M][blocks][128] and scales [M][blocks][1] in float32."""
    t = _padded(x.float(), 1).view(x.shape[0], -1, BLOCK)
    code = _scale_code(t.abs().amax(dim=2, keepdim=True))
    return (t * _power(254 - code)).to(torch.float8_e4m3fn).float(), _power(code)


def _rows_rounded(x):
    """x with every 128 values of a row rounded to 8 bits."""
    q, scale = _rows_quantised(x)
    return (q * scale).view(x.shape[0], -1)[:, :x.shape[1]]


def _weights_rounded(w, scale, k):
    """8-bit [..][N][K up to 128] with its block scales -> float32 [..][N][K]."""
    s = _power(scale).repeat_interleave(BLOCK, dim=-2)[..., :w.shape[-2], :].repeat_interleave(BLOCK, dim=-1)
    return (w.float() * s)[..., :k]


def _plain_product(s):
    c, ends = s["case"], s["ends"]
    spans = list(zip(ends[:-1], ends[1:]))
    w = _weights_rounded(s["w"], s["w_scale"], c["k"])
    a = _rows_rounded(s["x"])
    if c["gather"]:
        a = a[(s["pairs"] // c["gather"]).long()]
    y = torch.cat([a[i:j] @ w[g].t() for g, (i, j) in enumerate(spans)]).to(torch.bfloat16)
    if not c["train"]:
        return y
    d = _rows_rounded(s["dy"])
    dx = torch.cat([d[i:j] @ w[g] for g, (i, j) in enumerate(spans)]).to(torch.bfloat16)
    dy, x = s["dy"].float(), s["x"].float()      # the weight's gradient takes both as they are
    return y, dx, torch.stack([dy[i:j].t() @ x[i:j] for i, j in spans])


def _plain_layer(s):
    c = s["case"]
    ids, weights = _select(s["logits"], s["bias"], c["k"], c["groups"], c["topk_groups"])
    x, flat = s["x"].float(), ids.clamp(min=0).long().view(-1)
    widths = dict(gate=c["hidden"], up=c["hidden"], down=c["inter"])

    def rows(name, at):
        w, scale = s[name], s[name + "_scale"]
        if scale is None:
            return w[at].float()
        return _weights_rounded(w.view(torch.uint8)[at].view(w.dtype), scale[at], widths[name])

    if flat.numel() < c["experts"]:      # few pairs: each pair's own matrices
        xs = x.repeat_interleave(c["k"], dim=0)[:, :, None]
        gate, up = (torch.matmul(rows(name, flat), xs)[:, :, 0] for name in ("gate", "up"))
        y = torch.matmul(rows("down", flat), (F.silu(gate) * up)[:, :, None])[:, :, 0].view(*ids.shape, -1)
        out = (y * weights[:, :, None]).sum(dim=1)
    else:                                # many: every expert on every token
        every = torch.arange(c["experts"], device="cuda")
        gate, up = (torch.matmul(rows(name, every), x.t()) for name in ("gate", "up"))
        dense = torch.zeros((ids.shape[0], c["experts"]), device="cuda")
        dense.scatter_add_(1, ids.clamp(min=0).long(), weights)
        h = F.silu(gate) * up * dense.t()[:, None, :]
        out = torch.matmul(rows("down", every), h).sum(dim=0).t()
    return out.to(torch.bfloat16), ids, weights


def _noise(count, word):
    """Two words of 20 pseudo-random bits for each element, from its index and the tensor's word."""
    h = (torch.arange(count, device="cuda") + word) & 0xFFFFFFFF
    h = (h * MIX[0]) & 0xFFFFFFFF
    h = h ^ (h >> 15)
    h = (h * MIX[1]) & 0xFFFFFFFF
    h = h ^ (h >> 13)
    h = (h * MIX[2]) & 0xFFFFFFFF
    h = h ^ (h >> 16)
    return (h & 0xFFFFF).int(), (((h * MIX[0]) & 0xFFFFFFFF) >> 12).int()


def _state_scale(t):
    """The scale byte of each block: 2**(c - 127) with the block's largest value at most 1.875 times it."""
    bits = t.abs().amax(dim=1, keepdim=True).view(torch.int32)
    return ((bits >> 23) + ((bits & 0x7FFFFF) > 0x700000).int()).clamp(1, 253)


def _state_encode(x, noise, low, signed):
    """float32 -> (bytes, scale bytes): 3 bits of mantissa, rounded at random, `low` the code below the least one."""
    n = x.numel()
    t = F.pad(x, [0, -n % BLOCK]).view(-1, BLOCK)
    scale = _state_scale(t)
    bits = (t.abs() * _power(254 - scale)).view(-1)[:n].view(torch.int32)
    code = ((bits + noise) >> 20) - low
    if signed:
        code = code.clamp(0, 127) | ((x < 0).int() << 7)
    else:
        code = torch.where(x > 0, code.clamp(1, 255), 0)
    return code.to(torch.uint8), scale.view(-1).to(torch.uint8)


def _state_decode(q, scale, low, signed):
    code = q.int()
    mag = code & 127 if signed else code
    value = torch.where(mag > 0, ((mag + low) << 20).view(torch.float32), 0.0)
    value = value * _power(scale).repeat_interleave(BLOCK)[:q.numel()]
    return torch.where(code > 127, -value, value) if signed else value


M_LOW, V_LOW = 896, 768


def _plain_adamw(s):
    c = s["case"]
    s["step"] += 1
    t = s["step"]
    rate, root = LR / (1 - BETA1 ** t), 1 / math.sqrt(1 - BETA2 ** t)
    ms, vs = [], []

    def one(i, p, grad):
        g = grad.float()
        if c["bits"] == 32:
            m0, v0 = s["m"][i], s["v"][i]
        else:
            m0 = _state_decode(s["m"][i], s["m_scale"][i], M_LOW, True)
            v0 = _state_decode(s["v"][i], s["v_scale"][i], V_LOW, False)
        m = m0 * BETA1 + g * (1 - BETA1)
        v = v0 * BETA2 + (g * g) * (1 - BETA2)
        p.copy_(p * (1 - LR * DECAY) - rate * (m / (torch.sqrt(v) * root + EPS)))
        if c["copy"]:
            s["copies"][i].copy_(p)
        if c["bits"] == 32:
            m0.copy_(m)
            v0.copy_(v)
            return m0, v0
        rv, rm = _noise(p.numel(), (s["seed"] + t * MIX[0] + i * MIX[1]) & 0xFFFFFFFF)
        s["m"][i], s["m_scale"][i] = _state_encode(m, rm, M_LOW, True)
        s["v"][i], s["v_scale"][i] = _state_encode(v, rv, V_LOW, False)
        return (_state_decode(s["m"][i], s["m_scale"][i], M_LOW, True),
                _state_decode(s["v"][i], s["v_scale"][i], V_LOW, False))

    states = [one(i, p, g) for i, (p, g) in enumerate(zip(s["params"], s["grads"]))]
    ms, vs = [a for a, _ in states], [b for _, b in states]
    return dict(params=s["params"], m=ms, v=vs, copies=s["copies"])


def _plain(s):
    c = s["case"]
    if c["kind"] == "gate":
        ids, weights = _select(s["logits"], s["bias"], c["k"], c["groups"], c["topk_groups"])
        if not c["backward"]:
            return ids, weights
        d = weights * (s["grad"] - (weights * s["grad"]).sum(dim=1, keepdim=True))
        dl = torch.zeros(s["logits"].shape, device="cuda").scatter_add_(1, ids.clamp(min=0).long(), d)
        return ids, weights, dl.to(s["logits"].dtype)
    if c["kind"] == "product":
        return _plain_product(s)
    return _plain_layer(s) if c["kind"] == "layer" else _plain_adamw(s)


# ------------------------------------------------------------------------------------------------ the package's calls

def _own(s):
    import moe_expert_load_layer_amd as ep
    c = s["case"]
    if c["kind"] == "gate":
        ids, weights = ep.ep_gate_topk(s["logits"], c["k"], bias=s["bias"], num_groups=c["groups"],
                                       topk_groups=c["topk_groups"])
        if not c["backward"]:
            return ids, weights
        return ids, weights, ep.ep_gate_topk_backward(ids, weights, s["grad"], c["experts"], dtype=s["logits"].dtype)
    if c["kind"] == "product":
        xq, xs = ep.ep_quant_rows(s["x"])
        y = ep.ep_grouped_matmul(xq, xs, s["w"], s["w_scale"], s["offsets"], rows=s["pairs"],
                                 rows_div=max(1, c["gather"]))
        if not c["train"]:
            return y
        dq, ds = ep.ep_quant_rows(s["dy"])
        dx = ep.ep_grouped_matmul(dq, ds, s["wt"], s["wt_scale"], s["offsets"])
        return y, dx, ep.ep_grouped_wgrad(s["dy"], s["x"], s["offsets"])
    if c["kind"] == "layer":
        return ep.ep_moe_few_tokens(s["x"], s["logits"], c["k"], s["gate"], s["up"], s["down"], s["gate_scale"],
                                    s["up_scale"], s["down_scale"], bias=s["bias"], num_groups=c["groups"],
                                    topk_groups=c["topk_groups"])
    opt = s["opt"]
    opt.step(s["grads"], lr=LR)
    m, v = opt.states()
    return dict(params=s["params"], m=m, v=v, copies=s["copies"])


def run(state):
    return _own(state) if own else _plain(state)


# ------------------------------------------------------------------------------------------------ work

def work(case):
    c = case
    if c["kind"] == "gate":
        width = 4 if c["dtype"] == "float32" else 2
        scores, chosen = c["tokens"] * c["experts"], c["tokens"] * c["k"]
        return dict(bytes=scores * width * (2 if c["backward"] else 1) + chosen * (20 if c["backward"] else 8),
                    flops=scores * 2)
    if c["kind"] == "product":
        kp = -(-c["k"] // BLOCK) * BLOCK
        used = max(1, c["groups"] - (c["groups"] > 2)) if c["pairs"] >= 4 * c["groups"] else 1
        tokens = -(-c["pairs"] // c["gather"]) if c["gather"] else c["pairs"]
        w, x, y = used * c["n"] * kp, tokens * c["k"] * 2, c["pairs"] * c["n"] * 2
        ops = 2 * c["pairs"] * c["n"] * c["k"]
        if c["train"]:
            return dict(bytes=2 * w + 2 * x + 2 * y + 4 * c["groups"] * c["n"] * c["k"], flops=3 * ops)
        return dict(bytes=w + x + y, flops=ops)
    if c["kind"] == "layer":
        # distinct experts that tokens with such logits choose, over a few draws of the same law
        pairs, r, hits = c["tokens"] * c["k"], np.random.default_rng(1), []
        for _ in range(8):
            z = 1.5 * r.standard_normal((c["tokens"], c["experts"])) + np.exp(0.7 * r.standard_normal(c["experts"]))
            if c["masked"]:
                z = z[r.random(c["tokens"]) >= 0.1]
            if c["groups"] > 1:
                best = z.reshape(len(z), c["groups"], -1).max(axis=2)
                rank = np.argsort(np.argsort(-best, axis=1), axis=1)
                z = np.where(np.repeat(rank < c["topk_groups"], c["experts"] // c["groups"], axis=1), z, -np.inf)
            hits.append(len(np.unique(np.argsort(-z, axis=1)[:, :c["k"]])))
        hit = max(1.0, float(np.mean(hits)))
        each = 3 * c["hidden"] * c["inter"]
        return dict(bytes=hit * each * (2 if c["weights"] == "bfloat16" else 1) + 4 * c["tokens"] * c["hidden"],
                    flops=2 * pairs * each)
    n = c["tensors"] * c["size"]
    each = 8 + (4 if c["grads"] == "float32" else 2) + (16 if c["bits"] == 32 else 4 + 8) + (2 if c["copy"] else 0)
    return dict(bytes=n * each, flops=n * 15)


# ------------------------------------------------------------------------------------------------ 64 bits

def _exact_power(e):
    """2**e in float64, exactly, for whole numbers e."""
    return ((e.to(torch.int64) + 1023) << 52).view(torch.float64)


def _exact_round(t):
    """Float64 blocks of 128 along the last axis -> the 8-bit values they are held as, in float64."""
    amax = t.abs().amax(dim=-1, keepdim=True)
    mant, ex = torch.frexp(torch.where(amax > 0, amax, 1.0))
    unit = _exact_power((ex + torch.where(mant > 0.875, 1, 0) - 9).clamp(min=-126))
    v = t / unit
    step = _exact_power(torch.frexp(v.abs().clamp(min=2.0 ** -6)).exponent - 4)
    return torch.round(v / step) * step * unit


def _exact_rows(x):
    m, k = x.shape
    wide = torch.zeros((m, -(-k // 128) * 128), dtype=torch.float64, device=x.device)
    wide[:, :k] = x.double()
    return _exact_round(wide.view(m, -1, 128)).view(m, -1)[:, :k]


def _exact_weights(w, code, k):
    n = w.shape[0]
    unit = _exact_power(code.int() - 127)
    rows = torch.arange(n, device=w.device) // 128
    cols = torch.arange(w.shape[1], device=w.device) // 128
    return (w.double() * unit[rows][:, cols])[:, :k]


def _exact_choice(logits, bias, k, groups, topk_groups):
    score = (logits.float() + (0 if bias is None else bias)).cpu().numpy().astype(np.float64)
    l = logits.double().cpu().numpy()
    tokens, experts = score.shape
    if groups > 1:
        best = score.reshape(tokens, groups, -1).max(axis=2)
        order = np.argsort(-best, axis=1, kind="stable")
        rank = np.argsort(order, axis=1, kind="stable")
        score = np.where(np.repeat(rank < topk_groups, experts // groups, axis=1), score, -np.inf)
    ids = np.argsort(-score, axis=1, kind="stable")[:, :k]
    here = np.take_along_axis(score, ids, 1) > -np.inf
    z = np.where(here, np.take_along_axis(l, ids, 1), -np.inf)
    top = np.where(here.any(axis=1, keepdims=True), z.max(axis=1, keepdims=True), 0.0)
    e = np.where(here, np.exp(np.where(here, z - top, 0.0)), 0.0)
    total = e.sum(axis=1, keepdims=True)
    return np.where(here, ids, -1).astype(np.int32), e / np.where(total > 0, total, 1.0)


def _exact_state(x, noise, scale_at, floor, positive):
    """The value an 8-bit state holds for x: its magnitude cut to 3 bits of mantissa after the noise is added."""
    unit = _exact_power(scale_at - 127)
    mant, ex = torch.frexp((x.abs() / unit))
    place = _exact_power(ex - 4)
    cut = torch.floor(x.abs() / unit / place + noise.double() / 2 ** 20) * place
    least = 1.125 * 2.0 ** floor
    if positive:
        return torch.where(x > 0, cut.clamp(min=least, max=1.875), 0.0) * unit
    return torch.where(cut < least, 0.0, cut.clamp(max=1.875)) * unit * torch.sign(x)


def _exact_scale(x):
    n = x.numel()
    wide = torch.zeros(-(-n // 128) * 128, dtype=torch.float64, device=x.device)
    wide[:n] = x.abs().float().double()
    mant, ex = torch.frexp(wide.view(-1, 128).amax(dim=1))
    code = torch.where(mant > 0, ex + 126 + (mant > 0.9375).int(), 0).clamp(1, 253)
    return code.repeat_interleave(128)[:n]


def exact(case, seed):
    c, s = case, prepare(case, seed)
    if c["kind"] == "gate":
        ids, w = _exact_choice(s["logits"], s["bias"], c["k"], c["groups"], c["topk_groups"])
        if not c["backward"]:
            return ids, w
        g = s["grad"].double().cpu().numpy()
        d = np.where(ids >= 0, w * (g - (w * g).sum(axis=1, keepdims=True)), 0.0)
        dl = np.zeros((c["tokens"], c["experts"]))
        np.add.at(dl, (np.arange(c["tokens"])[:, None], np.maximum(ids, 0)), d)
        return ids, w, dl
    if c["kind"] == "product":
        a = _exact_rows(s["x"])
        y = torch.zeros((c["pairs"], c["n"]), dtype=torch.float64, device="cuda")
        dx = torch.zeros((c["pairs"], c["k"]), dtype=torch.float64, device="cuda")
        dw = torch.zeros((c["groups"], c["n"], c["k"]), dtype=torch.float64, device="cuda") if c["train"] else None
        d = _exact_rows(s["dy"]) if c["train"] else None
        for g in range(c["groups"]):
            i, j = s["ends"][g], s["ends"][g + 1]
            if i == j:
                continue
            w = _exact_weights(s["w"][g], s["w_scale"][g], c["k"])
            rows = a[(s["pairs"][i:j] // c["gather"]).long()] if c["gather"] else a[i:j]
            y[i:j] = rows @ w.t()
            if c["train"]:
                dx[i:j] = d[i:j] @ w
                dw[g] = s["dy"][i:j].double().t() @ s["x"][i:j].double()
        return (y, dx, dw) if c["train"] else y
    if c["kind"] == "layer":
        ids, w = _exact_choice(s["logits"], s["bias"], c["k"], c["groups"], c["topk_groups"])
        x = s["x"].double()
        out = torch.zeros_like(x)

        def matrix(name, e, k):
            return s[name][e].double() if s[name + "_scale"] is None else _exact_weights(
                s[name][e], s[name + "_scale"][e], k)

        for e in np.unique(ids[ids >= 0]):
            t, j = np.nonzero(ids == e)
            at = torch.from_numpy(t).cuda()
            gate = x[at] @ matrix("gate", e, c["hidden"]).t()
            h = gate / (1 + torch.exp(-gate)) * (x[at] @ matrix("up", e, c["hidden"]).t())
            out[at] += torch.from_numpy(w[t, j]).cuda()[:, None] * (h @ matrix("down", e, c["inter"]).t())
        return out, ids, w
    params, ms, vs, copies = [], [], [], []
    for i, (p, grad) in enumerate(zip(s["params"], s["grads"])):
        g = grad.double()
        m, v = (1 - BETA1) * g, (1 - BETA2) * g * g
        new = p.double() * (1 - LR * DECAY) - LR / (1 - BETA1) * m / (torch.sqrt(v / (1 - BETA2)) + EPS)
        params.append(new)
        copies.append(new)
        if c["bits"] == 8:
            rv, rm = _noise(p.numel(), (s["seed"] + MIX[0] + i * MIX[1]) & 0xFFFFFFFF)
            m = _exact_state(m, rm, _exact_scale(m), -15, False)
            v = _exact_state(v, rv, _exact_scale(v), -31, True)
        ms.append(m)
        vs.append(v)
    return dict(params=params, m=ms, v=vs, copies=copies if c["copy"] else None)
