"""Operators of a layer served in few bits: what one pass of each computes, in plain torch operations.

Four operators stand next to the sparse attention path and the layer around it:

* ``quantize``: bf16 activations -> E4M3 codes with one power-of-two scale per token and block of 128 channels;
* ``product``: the product of such activations with E4M3 weights that have one fp32 scale per 128 x 128 block;
* ``cache``: new latent rows written into the 4-bit latent cache at their positions, and those rows read back;
* ``attend``: the sparse latent attention over the selected rows of the 4-bit cache, with the head gate.

A row of the 4-bit cache is 416 bytes: 256 bytes of E2M1 codes (dims 2j and 2j + 1 in the low and high half of
byte j), 32 E4M3 scales (one for 16 dims), 64 bf16 rope values.

``run`` computes the plain form, or calls the package when ``own`` is set.  ``exact`` is the same in 64 bits.
"""
import math

import torch

own = False

HEADS, LATENT, ROPE = 64, 512, 64
ROW4 = 416  # bytes of one 4-bit cache row
SCALE = 192.0 ** -0.5
BLOCK = 128
GROUP = 16
MAX_WORK_ROWS = 512  # queries of the largest prefill block measured
STATUS_WS = 256  # bytes of the zero-filled workspace that a program keeps for the calls
E2M1 = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)
OUT_TYPES = {"bf16": torch.bfloat16, "fp32": torch.float32}


def listed():
    return [
        # one token's hidden state, quantised in front of the first projection
        {"name": "quantize 1 x 7168", "op": "quantize", "tokens": 1, "k": 7168},
        # a prefill chunk's attention output in front of the output projection
        {"name": "quantize 4096 x 8192", "op": "quantize", "tokens": 4096, "k": 8192},
        # decode of 4 sequences: hidden states through the packed first projection
        {"name": "product 4 x 2304 x 7168", "op": "product", "tokens": 4, "m": 2304, "k": 7168, "out": "fp32"},
        # decode of 32 sequences: the query projection
        {"name": "product 32 x 20544 x 1536", "op": "product", "tokens": 32, "m": 20544, "k": 1536, "out": "bf16"},
        # a ragged chunk through weights whose last blocks are partial
        {"name": "product 333 x 1111 x 1552", "op": "product", "tokens": 333, "m": 1111, "k": 1552, "out": "fp32"},
        # a prefill chunk through the output projection
        {"name": "product 4096 x 7168 x 8192", "op": "product", "tokens": 4096, "m": 7168, "k": 8192, "out": "bf16"},
        # decode of 32 sequences: one new row each
        {"name": "cache 32 x 1", "op": "cache", "batch": 32, "tokens": 1, "ctx": 8192},
        # a prefill chunk's rows
        {"name": "cache 1 x 4096", "op": "cache", "batch": 1, "tokens": 4096, "ctx": 32768},
        # decode of 4 sequences at 8K
        {"name": "attend 4 x 1, ctx 8192", "op": "attend", "batch": 4, "tokens": 1, "ctx": 8192, "top_k": 2048,
         "gate": True, "empty": False},
        # decode of 32 sequences at 128K
        {"name": "attend 32 x 1, ctx 131072", "op": "attend", "batch": 32, "tokens": 1, "ctx": 131072, "top_k": 2048,
         "gate": True, "empty": False},
        # short sequences whose selections are padded, one query with nothing selected, no gate
        {"name": "attend 3 x 5, ctx 1001, padded", "op": "attend", "batch": 3, "tokens": 5, "ctx": 1001, "top_k": 1088,
         "gate": False, "empty": True},
        # a prefill block late in a long context
        {"name": "attend 1 x 512, ctx 65536", "op": "attend", "batch": 1, "tokens": 512, "ctx": 65536, "top_k": 2048,
         "gate": True, "empty": False},
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(("quantize", "product", "product", "cache", "attend", "attend"))
    if op == "quantize":
        return {"op": op, "tokens": _log(rng, 1, 4096), "k": 16 * _log(rng, 1, 512)}
    if op == "product":
        return {"op": op, "tokens": _log(rng, 1, 4096), "m": _log(rng, 64, 7168), "k": 16 * _log(rng, 8, 512),
                "out": rng.choice(("bf16", "fp32"))}
    if op == "cache":
        batch = _log(rng, 1, 32)
        return {"op": op, "batch": batch, "tokens": _log(rng, 1, 4096 // batch), "ctx": _log(rng, 4096, 32768)}
    batch = _log(rng, 1, 32)
    return {"op": op, "batch": batch, "tokens": _log(rng, 1, MAX_WORK_ROWS // batch),
            "ctx": _log(rng, 512, 131072 if batch <= 8 else 32768), "top_k": 64 * rng.randint(1, 32),
            "gate": rng.random() < 0.7, "empty": rng.random() < 0.3}


# ------------------------------------------------------------------------------------------------ inputs
def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(int(seed))
    ws = torch.zeros(STATUS_WS, dtype=torch.uint8, device="cuda")
    make = {"quantize": _prepare_quantize, "product": _prepare_product, "cache": _prepare_cache,
            "attend": _prepare_attend}[case["op"]]
    return {"case": dict(case), "ws": ws, **make(case, g)}


def _normal(g, *shape):
    return torch.randn(shape, generator=g, device="cuda")


def _activations(g, tokens, k):
    """Hidden states: N(0, 1) channels, a few of them some hundred times larger, one token in 16 all zero."""
    x = _normal(g, tokens, k)
    x *= torch.where(torch.rand((1, k), generator=g, device="cuda") < 0.01, 300.0, 1.0)
    x *= torch.exp2(torch.randint(-6, 7, (tokens, 1), generator=g, device="cuda").float())
    zero = torch.rand((tokens, 1), generator=g, device="cuda") < 1 / 16
    zero[0] = False
    return x.masked_fill_(zero, 0.0).to(torch.bfloat16)


def _prepare_quantize(case, g):
    return {"x": _activations(g, case["tokens"], case["k"])}


def _prepare_product(case, g):
    tokens, m, k = case["tokens"], case["m"], case["k"]
    codes, scale = _quantize(_activations(g, tokens, k).float())
    w = _normal(g, m, k) * k ** -0.5
    kb, mb = -(-k // BLOCK), -(-m // BLOCK)
    pad = torch.zeros((mb * BLOCK, kb * BLOCK), device="cuda")
    pad[:m, :k] = w
    blocks = pad.view(mb, BLOCK, kb, BLOCK)
    w_scale = (blocks.abs().amax((1, 3)) / 448.0).clamp_min(1e-12)
    w8 = (blocks / w_scale[:, None, :, None]).clamp(-448, 448).view(mb * BLOCK, kb * BLOCK)[:m, :k]
    return {"x": codes, "x_scale": scale, "w": w8.to(torch.float8_e4m3fn).contiguous(), "w_scale": w_scale.contiguous()}


def _prepare_cache(case, g):
    batch, tokens, ctx = case["batch"], case["tokens"], case["ctx"]
    rows = _normal(g, batch, tokens, LATENT + ROPE)
    rows *= torch.exp2(torch.randint(-3, 4, (batch, tokens, 1), generator=g, device="cuda").float())
    start = torch.randint(0, ctx - tokens + 1, (batch, 1), generator=g, device="cuda")
    pos = (start + torch.arange(tokens, device="cuda")).to(torch.int32)
    return {"rows": rows.to(torch.bfloat16), "pos": pos,
            "cache": torch.zeros((batch, ctx, ROW4), dtype=torch.uint8, device="cuda")}


def _prepare_attend(case, g):
    batch, tokens, ctx, top_k = case["batch"], case["tokens"], case["ctx"], case["top_k"]
    cache = torch.empty((batch, ctx, ROW4), dtype=torch.uint8, device="cuda")
    for b in range(batch):
        cache[b] = _pack(_normal(g, ctx, LATENT + ROPE).to(torch.bfloat16))
    q = _normal(g, batch, tokens, HEADS, LATENT + ROPE).to(torch.bfloat16)
    gate = _normal(g, batch, tokens, HEADS).to(torch.bfloat16) if case["gate"] else None
    # query i of a sequence stands at position ctx - tokens + i and sees top_k distinct positions up to it
    pos = torch.arange(ctx - tokens, ctx, device="cuda").clamp_min(0)
    seen = (pos + 1).view(1, tokens, 1).double()
    slot = torch.arange(top_k, device="cuda", dtype=torch.float64)
    stride = (seen / top_k).clamp_min(1.0)
    u = torch.rand((batch, tokens, top_k), generator=g, device="cuda", dtype=torch.float64)
    idx = (slot * stride + u * (stride - 1.0)).floor()
    idx = torch.where(idx < seen, idx, -1.0).to(torch.int32)
    if case["empty"]:  # a query whose selection leaves nothing
        idx[batch - 1, tokens // 2] = -1
    return {"q": q, "cache": cache, "idx": idx.contiguous(), "gate": gate}


# ------------------------------------------------------------------------------------------------ plain forms
def _quantize(x):
    """fp32 [tokens, k] -> E4M3 codes and the power-of-two scales [tokens, ceil(k / 128)]: the smallest 2^e with
    max |x| <= 448 * 2^e over the block (1 for a block of zeros; e >= -126)."""
    tokens, k = x.shape
    kb = -(-k // BLOCK)
    blocks = torch.nn.functional.pad(x, (0, kb * BLOCK - k)).view(tokens, kb, BLOCK)
    amax = blocks.abs().amax(2)
    mant, expo = torch.frexp(amax)  # amax = mant * 2^expo, mant in [0.5, 1); 448 = 0.875 * 2^9
    e = (expo - 9 + (mant > 0.875).int()).clamp_min(-126)
    scale = torch.where(amax > 0, torch.ldexp(torch.ones_like(amax), e), 1.0)
    codes = (blocks / scale[..., None]).view(tokens, kb * BLOCK)[:, :k].to(torch.float8_e4m3fn)
    return codes.contiguous(), scale


def _product(x, x_scale, w, w_scale, out_type):
    k, m = x.shape[1], w.shape[0]
    xs = x.float() * x_scale.repeat_interleave(BLOCK, 1)[:, :k]
    ws = w.float() * w_scale.repeat_interleave(BLOCK, 0)[:m].repeat_interleave(BLOCK, 1)[:, :k]
    return (xs @ ws.T).to(out_type)


def _pack(rows):
    """bf16 rows [..., 576] -> cache rows [..., 416] (uint8)."""
    x = rows[..., :LATENT].float().unflatten(-1, (LATENT // GROUP, GROUP))
    scale = (x.abs().amax(-1) / 6.0).clamp_max(448.0).to(torch.float8_e4m3fn)
    s = scale.float()[..., None]
    a = torch.where(s > 0, x / s, 0.0)
    m = a.abs()
    code = ((m > 0.25).to(torch.uint8) + (m >= 0.75) + (m > 1.25) + (m >= 1.75) + (m > 2.5) + (m >= 3.5) + (m > 5.0))
    code = (code + 8 * torch.signbit(x)).flatten(-2).to(torch.uint8)
    rope = rows[..., LATENT:].contiguous().view(torch.uint8)
    return torch.cat((code[..., 0::2] + 16 * code[..., 1::2], scale.view(torch.uint8), rope), -1)


def _unpack(packed, dtype=torch.float32):
    """cache rows [..., 416] -> their values [..., 576]."""
    lut = torch.tensor(E2M1 + tuple(-v for v in E2M1), dtype=dtype, device=packed.device)
    byte = packed[..., : LATENT // 2]
    code = torch.stack((byte & 15, byte >> 4), -1).flatten(-2)
    scale = packed[..., LATENT // 2 : LATENT // 2 + LATENT // GROUP].contiguous().view(torch.float8_e4m3fn).to(dtype)
    latent = lut[code.int()].unflatten(-1, (LATENT // GROUP, GROUP)) * scale[..., None]
    rope = packed[..., LATENT // 2 + LATENT // GROUP :].contiguous().view(torch.bfloat16).to(dtype)
    return torch.cat((latent.flatten(-2), rope), -1)


def _attend(q, cache, idx, gate, dtype=torch.float32):
    batch, tokens = q.shape[:2]
    seen = idx >= 0
    b = torch.arange(batch, device=q.device).view(batch, 1, 1)
    rows = _unpack(cache[b, idx.clamp_min(0)], dtype).flatten(0, 1)  # [batch * tokens, top_k, 576]
    z = torch.bmm(q.to(dtype).flatten(0, 1), rows.transpose(1, 2)) * SCALE
    z = z.masked_fill(~seen.flatten(0, 1)[:, None], -math.inf)
    top = z.amax(-1, keepdim=True)
    p = torch.exp(z - torch.where(top > -math.inf, top, 0.0))
    o = torch.bmm(p, rows[..., :LATENT]) / p.sum(-1, keepdim=True).clamp_min(1e-30)
    if gate is not None:
        o = o / (1.0 + torch.exp(-gate.to(dtype).flatten(0, 1)))[..., None]
    return o.unflatten(0, (batch, tokens))


# ------------------------------------------------------------------------------------------------ one pass
def run(state):
    return _run_own(state) if own else _run_plain(state)


def _run_plain(s):
    case = s["case"]
    if case["op"] == "quantize":
        codes, scale = _quantize(s["x"].float())
        return {"codes": codes, "scale": scale}
    if case["op"] == "product":
        return {"y": _product(s["x"], s["x_scale"], s["w"], s["w_scale"], OUT_TYPES[case["out"]])}
    if case["op"] == "cache":
        b = torch.arange(case["batch"], device="cuda")[:, None]
        s["cache"][b, s["pos"]] = _pack(s["rows"])
        return {"rows": _unpack(s["cache"][b, s["pos"]]).to(torch.bfloat16)}
    return {"out": _attend(s["q"], s["cache"], s["idx"], s["gate"]).to(torch.bfloat16)}


def _run_own(s):
    import sparse_gated_attention_b200 as sga

    case = s["case"]
    if case["op"] == "quantize":
        codes, scale = sga.quantize_fp8(s["x"])
        return {"codes": codes, "scale": scale}
    if case["op"] == "product":
        return {"y": sga.gemm_fp8(s["x"], s["x_scale"], s["w"], s["w_scale"], out_dtype=OUT_TYPES[case["out"]],
                                  ws=s["ws"])}
    if case["op"] == "cache":
        sga.kv4_append(s["rows"], s["pos"], s["cache"], ws=s["ws"])
        return {"rows": sga.kv4_read(s["cache"], s["pos"], ws=s["ws"])}
    return {"out": sga.sparse_mla_attend_kv4(s["q"], s["cache"], s["idx"], s["gate"], ws=s["ws"])}


def work(case):
    """Inputs read once and outputs written once; the multiply-adds of the contractions."""
    if case["op"] == "quantize":
        n = case["tokens"] * case["k"]
        return {"bytes": 3 * n + 4 * case["tokens"] * -(-case["k"] // BLOCK), "flops": 2 * n}
    if case["op"] == "product":
        t, m, k = case["tokens"], case["m"], case["k"]
        kb = -(-k // BLOCK)
        return {"bytes": t * k + m * k + 4 * kb * (t + -(-m // BLOCK)) + t * m * (2 if case["out"] == "bf16" else 4),
                "flops": 2 * t * m * k}
    if case["op"] == "cache":  # rows in, packed rows written and read, values out
        n = case["batch"] * case["tokens"]
        return {"bytes": n * (2 * (LATENT + ROPE) * 2 + 2 * ROW4 + 4), "flops": 4 * n * LATENT}
    n = case["batch"] * case["tokens"]
    rows = min(n * min(case["top_k"], case["ctx"]), case["batch"] * case["ctx"])  # a row read by several queries, once
    return {"bytes": rows * ROW4 + n * (HEADS * (2 * LATENT + ROPE) * 2 + 4 * case["top_k"] + 2 * HEADS),
            "flops": 2 * n * min(case["top_k"], case["ctx"]) * HEADS * (2 * LATENT + ROPE)}


# ------------------------------------------------------------------------------------------------ in 64 bits
def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "quantize":
        return _exact_quantize(s["x"].double())
    if case["op"] == "product":
        return {"y": _exact_product(s)}
    if case["op"] == "cache":
        return {"rows": _exact_rows(s["rows"])}
    return {"out": _exact_attend(s)}


def _round_e4m3(v):
    """Nearest E4M3 value (ties to even) of |v| <= 448, in 64 bits: 3 mantissa bits, steps of 2^-9 below 2^-6."""
    _, expo = torch.frexp(v)
    step = torch.ldexp(torch.ones_like(v), (expo - 4).clamp_min(-9))
    return torch.round(v / step) * step


def _exact_quantize(x):
    tokens, k = x.shape
    codes = torch.empty_like(x)
    scales = []
    for k0 in range(0, k, BLOCK):
        part = x[:, k0 : k0 + BLOCK]
        top = part.abs().amax(1)
        e = torch.ceil(torch.log2(torch.where(top > 0, top, 448.0) / 448.0) - 1e-12).clamp_min(-126)
        scales.append(torch.exp2(e))
        codes[:, k0 : k0 + BLOCK] = _round_e4m3(part / scales[-1][:, None])
    return {"codes": codes, "scale": torch.stack(scales, 1)}


def _exact_product(s):
    x, w = s["x"].double(), s["w"].double()
    y = torch.zeros((x.shape[0], w.shape[0]), dtype=torch.float64, device="cuda")
    row_block = torch.arange(w.shape[0], device="cuda") // BLOCK
    for j in range(s["x_scale"].shape[1]):
        part = slice(j * BLOCK, (j + 1) * BLOCK)
        y += (x[:, part] @ w[:, part].T) * s["x_scale"][:, j, None].double() * s["w_scale"][row_block, j].double()
    return y


def _exact_rows(rows):
    x = rows.double()
    latent, out = x[..., :LATENT], x.clone()
    grid = torch.tensor(E2M1, dtype=torch.float64, device="cuda")
    for d in range(0, LATENT, GROUP):
        part = latent[..., d : d + GROUP]
        s = _round_e4m3((part.abs().amax(-1, keepdim=True) / 6.0).clamp_max(448.0))
        a = torch.where(s > 0, part / s, 0.0).abs().clamp_max(6.0)
        # the nearest of the eight magnitudes; of two equally near ones the one with the even code
        far = (a[..., None] - grid).abs() + torch.tensor([0.0, 1e-13] * 4, dtype=torch.float64, device="cuda")
        out[..., d : d + GROUP] = torch.sign(part) * grid[far.argmin(-1)] * s
    return out


def _exact_attend(s):
    q, idx, gate = s["q"].double(), s["idx"], s["gate"]
    out = torch.zeros((*q.shape[:3], LATENT), dtype=torch.float64, device="cuda")
    for b in range(q.shape[0]):
        values = _exact_values(s["cache"][b])
        for i in range(q.shape[1]):
            rows = values[idx[b, i][idx[b, i] >= 0].long()]
            if rows.shape[0]:
                p = torch.softmax(q[b, i] @ rows.T / 192.0 ** 0.5, -1)
                out[b, i] = p @ rows[:, :LATENT]
    return out if gate is None else out * torch.sigmoid(gate.double())[..., None]


def _exact_values(packed):
    """The values of one sequence's cache rows, in 64 bits (every one of them is a bf16 value)."""
    byte = packed[:, : LATENT // 2].to(torch.int32)
    code = torch.empty((packed.shape[0], LATENT), dtype=torch.int32, device="cuda")
    code[:, 0::2], code[:, 1::2] = byte % 16, byte // 16
    e, m = (code // 2) % 4, (code % 2).double()
    mag = torch.where(e > 0, torch.exp2(e.double() - 1.0) * (1.0 + m / 2.0), m / 2.0)
    raw = packed[:, LATENT // 2 : LATENT // 2 + LATENT // GROUP].to(torch.int32)
    se, sm = raw // 8, (raw % 8).double()
    scale = torch.where(se > 0, torch.exp2(se.double() - 7.0) * (1.0 + sm / 8.0), sm * 2.0 ** -9)
    latent = torch.where(code >= 8, -mag, mag) * scale.repeat_interleave(GROUP, 1)
    bits = packed[:, LATENT // 2 + LATENT // GROUP :].to(torch.int32)
    rope = ((bits[:, 0::2] + 256 * bits[:, 1::2]) << 16).view(torch.float32).double()
    return torch.cat((latent, rope), 1)
