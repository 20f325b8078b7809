"""What is measured of the prompt path's operators: rotary positions, attention over whole
packed prompts, and attention of ragged chunks over the compressed paged cache.

Each operator has a plain form here (elementary torch operations in 32 bits, angles in 64)
and the library's call; `own` chooses.  `exact` gives the results in 64 bits from the
definitions, written apart from the plain forms.  Sizes are those of the repository's
workloads (llama8b: 8 kv / 32 query heads; long70b: 8 / 64; batched: 32 sequences of 4096
tokens; head dimension 128; pages of 16 tokens) and ragged ones around them.
"""
import functools
import math

import numpy as np
import torch

own = False

D = 128
PAGE = 16

# ---------------------------------------------------------------- cases
# rope:   T tokens; rot rotated dimensions; far: largest position; fused: q and k are rows of one
#         projection [T][(Hq + 2 Hkv) 128] (token stride), else tensors of their own.
# prompt: lens: the packed sequences' lengths.
# chunk:  nq: new tokens of each sequence; ctx: its cached tokens, the new ones among them;
#         bits, rotation (0 Haar, 1 Hadamard), mode (0 keys with sign sketch, 1 without).


def listed():
    return [
        # one decode step of the batched workload: latency
        dict(name="rope decode step", op="rope", T=32, Hq=32, Hkv=8, rot=128, layout="half", scaling="none",
             factor=1.0, far=4200, fused=False),
        # a packed batch of prompts, half of each head rotated, positions interpolated
        dict(name="rope partial interleaved", op="rope", T=4099, Hq=32, Hkv=8, rot=64, layout="interleaved",
             scaling="linear", factor=4.0, far=16384, fused=False),
        # a long prompt out of a fused projection, ramped scaling
        dict(name="rope long prompt", op="rope", T=32768, Hq=64, Hkv=8, rot=128, layout="half", scaling="yarn",
             factor=8.0, far=131072, fused=True),
        # a handful of short chat turns: latency
        dict(name="prompt short turns", op="prompt", Hq=32, Hkv=8, lens="1,130,17,64"),
        # ordinary prompts packed together
        dict(name="prompt packed", op="prompt", Hq=32, Hkv=8, lens="1033,257,2047,129,1500,800,640,515"),
        # one long document
        dict(name="prompt long", op="prompt", Hq=64, Hkv=8, lens="8192"),
        # verification of four drafted tokens in four sequences: latency
        dict(name="chunk verify", op="chunk", Hq=32, Hkv=8, nq="4,4,4,4", ctx="1000,513,2047,16", bits=4, rotation=0,
             mode=0),
        # the batched workload, a few new tokens in each sequence
        dict(name="chunk batched", op="chunk", Hq=32, Hkv=8,
             nq=",".join(str(1 + (5 * i) % 8) for i in range(32)), ctx=",".join(str(4096 - 31 * i) for i in range(32)),
             bits=4, rotation=0, mode=0),
        # a follow-up question at the end of the long70b context
        dict(name="chunk long context", op="chunk", Hq=64, Hkv=8, nq="256", ctx="131072", bits=4, rotation=1, mode=0),
        # the second half of a llama8b prompt
        dict(name="chunk half prompt", op="chunk", Hq=32, Hkv=8, nq="2048", ctx="4096", bits=4, rotation=0, mode=0),
        # a scheduler's mixed step: single tokens beside pieces of prompts
        dict(name="chunk mixed step", op="chunk", Hq=32, Hkv=8, nq="1,1,700,1,33,1", ctx="3001,77,1900,4096,33,1",
             bits=3, rotation=0, mode=0),
        # plain codes of two bits, one query head per kv head
        dict(name="chunk two bits", op="chunk", Hq=8, Hkv=8, nq="16,100", ctx="8191,777", bits=2, rotation=1, mode=1),
    ]


def _spread(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["rope", "prompt", "chunk"])
    Hkv = rng.choice([1, 2, 4, 8])
    G = rng.choice([1, 2, 3, 4, 5, 7, 8])
    if op == "rope":
        return dict(op=op, T=_spread(rng, 1, 32768), Hq=Hkv * G, Hkv=Hkv, rot=rng.choice([32, 64, 80, 96, 128]),
                    layout=rng.choice(["half", "interleaved"]),
                    scaling=rng.choice(["none", "linear", "ntk", "bands", "yarn"]),
                    factor=round(rng.uniform(1.5, 16.0), 2), far=_spread(rng, 2048, 131072), fused=rng.random() < 0.5)
    if op == "prompt":
        B = _spread(rng, 1, 12)
        top = _spread(rng, 1, int(8192 / math.sqrt(B)))
        lens = [top] + [_spread(rng, 1, top) for _ in range(B - 1)]
        rng.shuffle(lens)
        return dict(op=op, Hq=Hkv * G, Hkv=Hkv, lens=",".join(map(str, lens)))
    B = _spread(rng, 1, 32)
    top = _spread(rng, 16, 131072 // B)
    most = _spread(rng, 1, max(1, min(top, 2048, int(1.5e8 / (top * B * G)))))
    ctx = [top] + [_spread(rng, 1, top) for _ in range(B - 1)]
    nq = [min(c, _spread(rng, 1, most)) for c in ctx]
    return dict(op=op, Hq=Hkv * G, Hkv=Hkv, nq=",".join(map(str, nq)), ctx=",".join(map(str, ctx)),
                bits=rng.choice([2, 3, 4]), rotation=rng.choice([0, 1]), mode=rng.choice([0, 1]))


def _ints(text):
    return [int(x) for x in text.split(",")]


def _key_bits(case):
    return case["bits"] - 1 if case["mode"] == 0 else case["bits"]


def _width(b):
    return 4 if b >= 3 else b


def work(case):
    heads = case["Hq"] + case["Hkv"]
    if case["op"] == "rope":
        return {"bytes": case["T"] * (heads * D * 4 + 4), "flops": case["T"] * heads * case["rot"] * 3}
    if case["op"] == "prompt":
        lens = _ints(case["lens"])
        pairs = sum(n * (n + 1) // 2 for n in lens)
        return {"bytes": sum(lens) * (2 * case["Hq"] + 2 * case["Hkv"]) * D * 2, "flops": 4 * D * case["Hq"] * pairs}
    nq, ctx = _ints(case["nq"]), _ints(case["ctx"])
    pairs = sum(n * (c - n) + n * (n + 1) // 2 for n, c in zip(nq, ctx))
    row = D * _width(_key_bits(case)) // 8 + 4 + (D // 8 + 4 if case["mode"] == 0 else 0)
    row += D * _width(case["bits"]) // 8 + 4
    return {"bytes": sum(ctx) * case["Hkv"] * row + sum(nq) * case["Hq"] * D * 4, "flops": 4 * D * case["Hq"] * pairs}


# ---------------------------------------------------------------- the cache's parameters, from their seed
def _words(seed, tag, n):
    with np.errstate(over="ignore"):
        z = np.uint64(seed) + (np.uint64(tag) << np.uint64(48))
        z = z + np.arange(1, n + 1, dtype=np.uint64) * np.uint64(0x9E3779B97F4A7C15)
        z = (z ^ (z >> np.uint64(30))) * np.uint64(0xBF58476D1CE4E5B9)
        z = (z ^ (z >> np.uint64(27))) * np.uint64(0x94D049BB133111EB)
        return z ^ (z >> np.uint64(31))


def _levels(bits):
    """Lloyd-Max quantizer of N(0, 1): levels and the boundaries between them."""
    tail = lambda x: 0.5 * math.erfc(x / math.sqrt(2.0))  # noqa: E731
    dens = lambda x: math.exp(-0.5 * x * x) / math.sqrt(2.0 * math.pi)  # noqa: E731
    m = (1 << bits) // 2
    a = [3.0 * (k + 0.5) / m for k in range(m)]
    while True:
        e = [0.0] + [0.5 * (a[k - 1] + a[k]) for k in range(1, m)] + [math.inf]
        b = [(dens(e[k]) - dens(e[k + 1])) / (tail(e[k]) - tail(e[k + 1])) for k in range(m)]
        off, a = max(abs(x - y) for x, y in zip(a, b)), b
        if off < 1e-15:
            break
    c = np.array([-x for x in reversed(a)] + a)
    t = 0.5 * (c[1:] + c[:-1])
    t[m - 1] = 0.0
    return c, t


@functools.lru_cache(maxsize=None)
def _params(seed, bits, rotation, mode):
    if rotation == 0:
        u = ((_words(seed, 0, D * D) >> np.uint64(11)).astype(np.float64) + 0.5) * 2.0 ** -53
        rho, ang = np.sqrt(-2.0 * np.log(u[0::2])), 2.0 * np.pi * u[1::2]
        g = np.stack([rho * np.cos(ang), rho * np.sin(ang)], 1).reshape(D, D)
        Q, U = np.linalg.qr(g)
        R = Q * np.sign(np.diag(U))
    else:
        sign = np.where(_words(seed, 2, D) >> np.uint64(63), -1.0, 1.0)
        i = np.arange(D)
        H = np.array([[-1.0 if bin(x & y).count("1") & 1 else 1.0 for y in i] for x in i])
        R = (H * sign / math.sqrt(D)).T.copy()
    S = np.where(_words(seed, 1, D * D) >> np.uint64(63), -1.0, 1.0).reshape(D, D)
    cv, tv = _levels(bits)
    ck, tk = _levels(bits - 1 if mode == 0 else bits)
    return {k: torch.as_tensor(v) for k, v in dict(R=R, S=S, cv=cv, tv=tv, ck=ck, tk=tk).items()}


PARAM_SEED = 7


def _case_params(case):
    return _params(PARAM_SEED, case["bits"], case["rotation"], case["mode"])


# ---------------------------------------------------------------- inputs
def _gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def _normal(g, *shape):
    return torch.randn(shape, generator=g, device="cuda")


def _channel_law(g, Hkv):
    """Per-channel scales with a few loud channels, as keys and values have them."""
    s = torch.exp(0.5 * _normal(g, Hkv, D))
    loud = torch.rand((Hkv, D), generator=g, device="cuda").argsort(dim=1)[:, :3]
    return s * (1.0 + 7.0 * torch.zeros_like(s).scatter(1, loud, 1.0))


def _pack(codes, width):
    per = 8 // width
    c = codes.reshape(*codes.shape[:-1], D // per, per).to(torch.int32)
    return (c << (width * torch.arange(per, device="cuda", dtype=torch.int32))).sum(-1).to(torch.uint8)


def _bytes_of(x):
    return x.to(torch.float32).contiguous().unsqueeze(-1).view(torch.uint8).reshape(*x.shape, 4)


def _compressed(x, case, P, kind):
    """The packed fields of rows x [..., 128] (float32 values of fp16), by field."""
    R, S = P["R"].to("cuda", torch.float32), P["S"].to("cuda", torch.float32)
    c, t = (P["ck"], P["tk"]) if kind == 0 else (P["cv"], P["tv"])
    bits = _key_bits(case) if kind == 0 else case["bits"]
    n = x.norm(dim=-1)
    v = (x @ R) * (math.sqrt(D) / n.clamp_min(1e-30)).unsqueeze(-1)
    codes = torch.bucketize(v, t.to("cuda", torch.float32))
    fields = [_pack(codes, _width(bits))]
    if kind == 0 and case["mode"] == 0:
        r = x - (n / math.sqrt(D)).unsqueeze(-1) * (c.to("cuda", torch.float32)[codes] @ R.T)
        fields += [_pack((r @ S.T >= 0).to(torch.int32), 1), _bytes_of(n), _bytes_of(r.norm(dim=-1))]
    else:
        fields += [_bytes_of(n)]
    return fields


def _rope_inputs(case, g):
    T, Hq, Hkv = case["T"], case["Hq"], case["Hkv"]
    if case["fused"]:
        x = _normal(g, T, (Hq + 2 * Hkv) * D).to(torch.float16)
        q, k = x[:, :Hq * D].view(T, Hq, D), x[:, Hq * D:(Hq + Hkv) * D].view(T, Hkv, D)
    else:
        q, k = _normal(g, T, Hq, D).to(torch.float16), _normal(g, T, Hkv, D).to(torch.float16)
    pos = torch.randint(0, case["far"], (T,), generator=g, device="cuda", dtype=torch.int32)
    return dict(q=q, k=k, pos=pos)


def _starts(lens):
    return torch.tensor([0] + list(np.cumsum(lens)), dtype=torch.int32, device="cuda")


def _prompt_inputs(case, g):
    lens = _ints(case["lens"])
    T, Hq, Hkv = sum(lens), case["Hq"], case["Hkv"]
    q = _normal(g, T, Hq, D).to(torch.float16)
    k = (_normal(g, T, Hkv, D) * _channel_law(g, Hkv)).to(torch.float16)
    v = (_normal(g, T, Hkv, D) * _channel_law(g, Hkv)).to(torch.float16)
    return dict(q=q, k=k, v=v, starts=_starts(lens))


def _chunk_inputs(case, g):
    nq, ctx = _ints(case["nq"]), _ints(case["ctx"])
    B, Hq, Hkv, P = len(nq), case["Hq"], case["Hkv"], _case_params(case)
    pages = (max(ctx) + PAGE - 1) // PAGE
    need = sum((c + PAGE - 1) // PAGE for c in ctx)
    nb = need + 3
    where = torch.randperm(nb, generator=g, device="cuda")
    c = torch.tensor(ctx, device="cuda")
    per = (c + PAGE - 1) // PAGE
    col = torch.arange(pages, device="cuda")
    table = torch.where(col < per[:, None], where[((per.cumsum(0) - per)[:, None] + col).clamp(max=nb - 1)], 0)
    caches = []
    for kind in (0, 1):
        # a page's rows that no token has written hold whatever was there
        x = (_normal(g, nb, PAGE, Hkv, D) * _channel_law(g, Hkv)).to(torch.float16).to(torch.float32).transpose(1, 2)
        f = [y.reshape(nb, Hkv, -1) for y in _compressed(x, case, P, kind)]
        caches.append(torch.cat(f, 2).contiguous())
    q = (_normal(g, sum(nq), Hq, D) / math.sqrt(D) * 2.0).to(torch.float16)
    return dict(q=q, kc=caches[0], vc=caches[1], table=table.to(torch.int32).contiguous(), starts=_starts(nq),
                lens=c.to(torch.int32), top=max(ctx), nmax=max(nq))


@functools.lru_cache(maxsize=None)
def _context(bits, rotation, mode):
    from kv_cache_vector_02_b200 import tq
    return tq.tq_init(D, bits, PARAM_SEED, rotation, mode)


def _plan(case):
    from kv_cache_vector_02_b200 import tq
    layout = tq.ROPE_HALF if case["layout"] == "half" else tq.ROPE_INTERLEAVED
    scaling = {"none": tq.ROPE_SCALE_NONE, "linear": tq.ROPE_SCALE_LINEAR, "ntk": tq.ROPE_SCALE_NTK,
               "bands": tq.ROPE_SCALE_BANDS, "yarn": tq.ROPE_SCALE_YARN}[case["scaling"]]
    return tq.tq_rope_plan(case["rot"], layout, ROPE_BASE, scaling, case["factor"], ROPE_ORIGINAL,
                           *ROPE_BETWEEN.get(case["scaling"], (0.0, 0.0)))


def prepare(case, seed):
    g = _gen(seed)
    s = {"rope": _rope_inputs, "prompt": _prompt_inputs, "chunk": _chunk_inputs}[case["op"]](case, g)
    s["case"] = case
    if own:
        from kv_cache_vector_02_b200 import tq
        s["out"] = torch.empty(s["q"].shape, dtype=torch.float16, device="cuda")
        if case["op"] == "rope":
            s["plan"] = _plan(case)
            s["k_out"] = torch.empty(s["k"].shape, dtype=torch.float16, device="cuda")
        else:
            s["ctx"] = _context(case.get("bits", 4), case.get("rotation", 0), case.get("mode", 0))
        if case["op"] == "chunk":
            n = tq.tq_chunk_workspace_bytes(s["ctx"], len(s["lens"]), s["q"].shape[0], case["Hq"], case["Hkv"], s["top"])
            s["workspace"] = torch.empty(n, dtype=torch.uint8, device="cuda")
    return s


# ---------------------------------------------------------------- plain forms
ROPE_BASE = 500000.0
ROPE_ORIGINAL = 8192
ROPE_BETWEEN = {"bands": (1.0, 4.0), "yarn": (1.0, 32.0)}


def _rope_freqs(case):
    """Scaled frequencies in radians a position, and the factor on rotated values."""
    rot, f, kind = case["rot"], case["factor"], case["scaling"]
    i = torch.arange(rot // 2, device="cuda", dtype=torch.float64)
    th = ROPE_BASE ** (-2.0 * i / rot)
    if kind == "linear":
        return th / f, 1.0
    if kind == "ntk":
        return (ROPE_BASE * f ** (rot / (rot - 2.0))) ** (-2.0 * i / rot), 1.0
    if kind == "bands":
        low, high = ROPE_BETWEEN[kind]
        keep = ((ROPE_ORIGINAL * th / (2.0 * math.pi) - low) / (high - low)).clamp(0.0, 1.0)
        return th * (keep + (1.0 - keep) / f), 1.0
    if kind == "yarn":
        slow, fast = ROPE_BETWEEN[kind]
        at = lambda b: rot * math.log(ROPE_ORIGINAL / (2.0 * math.pi * b)) / (2.0 * math.log(ROPE_BASE))  # noqa: E731
        lo, hi = max(math.floor(at(fast)), 0), min(math.ceil(at(slow)), rot - 1)
        ramp = ((i - lo) / max(hi - lo, 0.001)).clamp(0.0, 1.0)
        return th * (1.0 - ramp + ramp / f), 0.1 * math.log(f) + 1.0
    return th, 1.0


def _plain_rope(s):
    case = s["case"]
    rot = case["rot"]
    th, m = _rope_freqs(case)
    a = s["pos"].to(torch.float64)[:, None, None] * th
    co, si = (m * torch.cos(a)).float(), (m * torch.sin(a)).float()
    half = case["layout"] == "half"

    def turned(x):
        x = x.float()
        r = x[..., :rot].unflatten(-1, (2, rot // 2) if half else (rot // 2, 2))
        x1, x2 = r.unbind(-2 if half else -1)
        y = torch.stack([x1 * co - x2 * si, x2 * co + x1 * si], -2 if half else -1).flatten(-2)
        return torch.cat([y, x[..., rot:]], -1).to(torch.float16)

    return turned(s["q"]), turned(s["k"])


def _attend(q, k, v, last, live):
    """softmax attention: q [B, n, Hq, D]; k, v [B, L, Hkv, D]; query (b, i) sees keys j <= last[b, i]; rows of `live` count."""
    B, n, Hq, _ = q.shape
    L, Hkv = k.shape[1], k.shape[2]
    j = torch.arange(L, device="cuda")
    k = torch.where((j <= last[:, -1:])[..., None, None], k, 0.0)
    v = torch.where((j <= last[:, -1:])[..., None, None], v, 0.0)
    q = q.reshape(B, n, Hkv, Hq // Hkv, D).permute(0, 2, 3, 1, 4).reshape(B, Hkv, -1, D)
    s = (q / math.sqrt(D)) @ k.permute(0, 2, 3, 1)
    hide = (j > last[..., None])[:, None, None]
    s = s.view(B, Hkv, Hq // Hkv, n, L).masked_fill_(hide, -math.inf).view(B, Hkv, -1, L)
    s -= s.amax(-1, keepdim=True)
    s.exp_()
    o = (s @ v.transpose(1, 2)) / s.sum(-1, keepdim=True)
    o = o.view(B, Hkv, Hq // Hkv, n, D).permute(0, 3, 1, 2, 4).reshape(B, n, Hq, D)
    return o[live].to(torch.float16)


def _padded(starts, n):
    """Row numbers [B, n] of packed sequences padded at their ends, and which of them are rows."""
    i = torch.arange(n, device="cuda")
    size = (starts[1:] - starts[:-1]).long()
    live = i < size[:, None]
    return torch.where(live, starts[:-1, None].long() + i, starts[:-1, None].long()), live, size


def _plain_prompt(s):
    lens = _ints(s["case"]["lens"])
    rows, live, size = _padded(s["starts"], max(lens))
    last = torch.minimum(torch.arange(max(lens), device="cuda"), size[:, None] - 1)
    return _attend(s["q"][rows].float(), s["k"][rows].float(), s["v"][rows].float(), last, live)


def _unpack(b, width):
    per = 8 // width
    sh = width * torch.arange(per, device="cuda", dtype=torch.int32)
    return ((b.to(torch.int32).unsqueeze(-1) >> sh) & ((1 << width) - 1)).flatten(-2)


def _decoded(cache, table, case, P, kind):
    """Rows [B, tokens, Hkv, 128] of the pages in `table`, float32."""
    ch = cache[table.long()]  # [B, pages, Hkv, bytes]
    B, pages, Hkv, _ = ch.shape
    bits = _key_bits(case) if kind == 0 else case["bits"]
    row = D * _width(bits) // 8
    R = P["R"].to("cuda", torch.float32)
    c = (P["ck"] if kind == 0 else P["cv"]).to("cuda", torch.float32)
    floats = lambda x: x.contiguous().view(torch.float32).unsqueeze(-1)  # noqa: E731
    at = PAGE * row
    sketch = kind == 0 and case["mode"] == 0
    n0 = at + (PAGE * D // 8 if sketch else 0)
    codes = _unpack(ch[..., :at].reshape(B, pages, Hkv, PAGE, row), _width(bits))
    x = (c[codes] @ R.T) * (floats(ch[..., n0:n0 + 4 * PAGE]) / math.sqrt(D))
    if sketch:
        S = P["S"].to("cuda", torch.float32)
        sg = _unpack(ch[..., at:n0].reshape(B, pages, Hkv, PAGE, D // 8), 1).float() * 2.0 - 1.0
        x += (sg @ S) * (floats(ch[..., n0 + 4 * PAGE:n0 + 8 * PAGE]) * (math.sqrt(math.pi / 2.0) / D))
    return x.transpose(2, 3).reshape(B, pages * PAGE, Hkv, D)


def _plain_chunk(s):
    case, P = s["case"], _case_params(s["case"])
    k, v = (_decoded(s[c], s["table"], case, P, kind) for kind, c in enumerate(("kc", "vc")))
    rows, live, size = _padded(s["starts"], s["nmax"])
    first = s["lens"].long()[:, None] - size[:, None]
    last = torch.minimum(first + torch.arange(s["nmax"], device="cuda"), s["lens"].long()[:, None] - 1)
    return _attend(s["q"][rows].float(), k[:, :s["top"]], v[:, :s["top"]], last, live)


def run(s):
    op = s["case"]["op"]
    if not own:
        return {"rope": _plain_rope, "prompt": _plain_prompt, "chunk": _plain_chunk}[op](s)
    from kv_cache_vector_02_b200 import tq
    if op == "rope":
        tq.tq_rope(s["plan"], s["q"], s["k"], s["pos"], s["out"], s["k_out"])
        return s["out"], s["k_out"]
    if op == "prompt":
        tq.tq_prompt_attention(s["ctx"], s["q"], s["k"], s["v"], s["starts"], s["out"])
        return s["out"]
    tq.tq_chunk_attention(s["ctx"], s["q"], s["starts"], s["kc"], s["vc"], s["table"], s["lens"], s["top"], s["out"],
                          s["workspace"])
    return s["out"]


# ---------------------------------------------------------------- the definitions in 64 bits
def _exact_rope(s, case):
    rot, kind, f = case["rot"], case["scaling"], case["factor"]
    low, high = ROPE_BETWEEN.get(kind, (0.0, 0.0))
    corr = [rot * math.log(ROPE_ORIGINAL / (2 * math.pi * b)) / (2 * math.log(ROPE_BASE)) if b else 0 for b in (high, low)]
    lo, hi = max(math.floor(corr[0]), 0), min(math.ceil(corr[1]), rot - 1)
    m = 0.1 * math.log(f) + 1.0 if kind == "yarn" else 1.0
    out = [s["q"].double().clone(), s["k"].double().clone()]
    pos = s["pos"].double()[:, None]
    for i in range(rot // 2):
        th = ROPE_BASE ** (-2.0 * i / rot)
        if kind == "linear":
            th /= f
        elif kind == "ntk":
            th = (ROPE_BASE * f ** (rot / (rot - 2.0))) ** (-2.0 * i / rot)
        elif kind == "bands":
            wave = 2 * math.pi / th
            if wave > ROPE_ORIGINAL / low:
                th /= f
            elif wave > ROPE_ORIGINAL / high:
                u = (ROPE_ORIGINAL / wave - low) / (high - low)
                th = (1 - u) * th / f + u * th
        elif kind == "yarn":
            u = min(max((i - lo) / max(hi - lo, 0.001), 0.0), 1.0)
            th = u * th / f + (1 - u) * th
        a, b = (i, i + rot // 2) if case["layout"] == "half" else (2 * i, 2 * i + 1)
        ang = pos * th
        for x, y in zip((s["q"], s["k"]), out):
            xa, xb = x[..., a].double(), x[..., b].double()
            y[..., a] = m * (xa * torch.cos(ang) - xb * torch.sin(ang))
            y[..., b] = m * (xa * torch.sin(ang) + xb * torch.cos(ang))
    return tuple(out)


def _exact_rows(q, k, v, first):
    """q [n, Hq, D], k, v [L, Hkv, D] in 64 bits; query i sees keys 0 .. first + i."""
    n, Hq, _ = q.shape
    G = Hq // k.shape[1]
    out = torch.empty_like(q)
    for h in range(Hq):
        s = torch.einsum("id,jd->ij", q[:, h], k[:, h // G]) * D ** -0.5
        s = s.tril(first) + torch.full_like(s, -math.inf).triu(first + 1)
        out[:, h] = torch.softmax(s, 1) @ v[:, h // G]
    return out


def _exact_prompt(s, case):
    parts = [x.double().split(_ints(case["lens"])) for x in (s["q"], s["k"], s["v"])]
    return torch.cat([_exact_rows(q, k, v, 0) for q, k, v in zip(*parts)])


def _exact_cache(chunks, case, P, kind):
    """[pages, Hkv, bytes] -> the rows of these pages in 64 bits, [pages * 16, Hkv, 128]."""
    n, Hkv, _ = chunks.shape
    w = _width(_key_bits(case) if kind == 0 else case["bits"])
    c = (P["ck"] if kind == 0 else P["cv"]).cuda()
    bits = torch.stack([(chunks >> i) & 1 for i in range(8)], -1).flatten(2)  # one bit a value
    code_bits = bits[..., :PAGE * D * w].reshape(n, Hkv, PAGE, D, w).long()
    code = sum(code_bits[..., i] << i for i in range(w))
    at = PAGE * D * w // 8
    sketch = kind == 0 and case["mode"] == 0
    sg = bits[..., 8 * at:8 * at + PAGE * D].reshape(n, Hkv, PAGE, D).double() * 2 - 1 if sketch else None
    scal = chunks[..., at + (PAGE * D // 8 if sketch else 0):].contiguous().view(torch.float32).double()
    scal = scal.reshape(n, Hkv, -1, PAGE)
    x = torch.einsum("phtj,ij->phti", c[code], P["R"].cuda()) * scal[:, :, 0, :, None] / D ** 0.5
    if sketch:
        x += torch.einsum("phtj,ji->phti", sg, P["S"].cuda()) * scal[:, :, 1, :, None] * (math.pi / 2) ** 0.5 / D
    return x.permute(0, 2, 1, 3).reshape(n * PAGE, Hkv, D)


def _exact_chunk(s, case):
    P, out, at = _case_params(case), [], 0
    for b, (n, L) in enumerate(zip(_ints(case["nq"]), _ints(case["ctx"]))):
        pages = s["table"][b, :(L + PAGE - 1) // PAGE].long()
        k, v = (_exact_cache(s[c][pages], case, P, kind)[:L] for kind, c in enumerate(("kc", "vc")))
        out.append(_exact_rows(s["q"][at:at + n].double(), k, v, L - n))
        at += n
    return torch.cat(out)


def exact(case, seed):
    s = prepare(case, seed)
    return {"rope": _exact_rope, "prompt": _exact_prompt, "chunk": _exact_chunk}[case["op"]](s, case)
