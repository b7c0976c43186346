"""The block-scaled 8-bit path as measured work: the operators between two
Linears whose E4M3 activations carry one float32 scale for every 128 columns of
a row (`add_rmsnorm_fp8_block`, `gated_act_fp8_block`, `quantize_fp8_block`) and
the Linear on such activations and on weights with one scale for every 128 x 128
block (`linear_fp8_block`).

Each case is one call on inputs of a layer.  `run` computes it either through
the library (`own`) or in plain torch operations; `exact` computes it again in
float64 from the definition.
"""
import torch

own = False

E4M3_MAX = 448.0
BLOCK = 128
LEAST_SCALE = 2.0 ** -100          # the scale of a block of zeros


# ------------------------------------------------------------------- cases

def listed():
    return [
        # the gated AdaRMSNorm in front of a decode batch's Linear: latency
        dict(name="norm_decode", op="norm", rows=32, hidden=4096, mode="ada", gated=True),
        # a packed batch of odd length, a width whose last block is cut short
        dict(name="norm_odd", op="norm", rows=777, hidden=2736, mode="weight", gated=False),
        # prompts, wide model: bandwidth; the weight is folded into the Linear behind
        dict(name="norm_prefill", op="norm", rows=16384, hidden=8192, mode="noweight", gated=False),
        # a decode batch's SwiGLU
        dict(name="gated_decode", op="gated", rows=32, d=11008, act="silu"),
        # a prompt's SwiGLU
        dict(name="gated_prefill", op="gated", rows=4096, d=11008, act="silu"),
        # the attention's output in front of its projection, one prompt
        dict(name="quantize_attention", op="quantize", rows=4096, d=4096, block_rows=1),
        # a Linear's weight at load time
        dict(name="quantize_weight", op="quantize", rows=16384, d=4096, block_rows=128),
        # one request's token through a square projection: latency
        dict(name="linear_one_token", op="linear", m=1, n=4096, k=4096, act="none", bias=False),
        # a decode batch through the up projection with bias and GELU: reading the weight
        dict(name="linear_decode", op="linear", m=32, n=16384, k=4096, act="gelu_tanh", bias=True),
        # a packed batch of odd length through the down projection
        dict(name="linear_odd", op="linear", m=333, n=4096, k=11008, act="none", bias=False),
        # a chunk of a prompt through a square projection
        dict(name="linear_chunk", op="linear", m=1024, n=4096, k=4096, act="none", bias=True),
        # prompts through the up projection with bias and GELU: the largest
        dict(name="linear_prefill", op="linear", m=8192, n=16384, k=4096, act="gelu_tanh", bias=True),
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(lo * (hi / lo) ** rng.random()))))


def _width(rng, lo, hi):
    """A row's width: a multiple of 16, half of them whole blocks of 128."""
    step = rng.choice([16, 128])
    return step * _log_int(rng, max(1, lo // step), hi // step)


def draw(rng):
    op = rng.choice(["norm", "gated", "quantize", "linear", "linear", "linear"])
    if op == "norm":
        hidden = _width(rng, 64, 32768)
        return dict(op=op, rows=_log_int(rng, 1, min(65536, 16384 * 8192 // hidden)), hidden=hidden,
                    mode=rng.choice(["weight", "weight", "noweight", "ada"]), gated=rng.random() < 0.4)
    if op == "gated":
        d = _width(rng, 64, 32768)
        return dict(op=op, rows=_log_int(rng, 1, min(65536, 16384 * 8192 // d)), d=d,
                    act=rng.choice(["silu", "silu", "gelu_tanh", "gelu_erf"]))
    if op == "quantize":
        d = _width(rng, 16, 32768)
        return dict(op=op, rows=_log_int(rng, 1, min(65536, 16384 * 8192 // d)), d=d,
                    block_rows=rng.choice([1, 1, 128]))
    n, k = 8 * _log_int(rng, 8, 4096), _width(rng, 128, 16384)
    most = max(1, min(16384, (8192 * 16384 * 4096) // (n * k)))
    return dict(op=op, m=_log_int(rng, 1, most), n=n, k=k,
                act=rng.choice(["none", "none", "gelu_tanh", "gelu_erf", "silu"]), bias=rng.random() < 0.5)


# ------------------------------------------------------------------ inputs

def _blocks(n):
    return -(-n // BLOCK)


def _generator(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def _randn(g, *shape):
    return torch.randn(*shape, generator=g, device="cuda")


def _with_outliers(x, g, share=0.002, by=20.0):
    """`x` with a few columns that are much larger than the others, as activations have."""
    strong = torch.rand(x.shape[-1], generator=g, device="cuda") < share
    return x * torch.where(strong, by, 1.0)


def _prepare_norm(c, seed):
    g = _generator(seed)
    rows, h = c["rows"], c["hidden"]
    s = dict(x=_with_outliers(_randn(g, rows, h), g).bfloat16(), res=(_randn(g, rows, h) * 2).bfloat16(), eps=1e-6,
             weight=None, gate=None, ada_scale=None, ada_shift=None)
    if c["mode"] == "weight":
        s["weight"] = (1 + 0.1 * _randn(g, h)).bfloat16()
    if c["mode"] == "ada":
        s["ada_scale"], s["ada_shift"] = (0.2 * _randn(g, h)).bfloat16(), (0.2 * _randn(g, h)).bfloat16()
    if c["gated"]:
        s["gate"] = (0.2 * _randn(g, h)).bfloat16()
    return dict(s, res_out=torch.empty_like(s["x"]), q=torch.empty(rows, h, dtype=torch.uint8, device="cuda"),
                scales=torch.empty(rows, _blocks(h), device="cuda"))


def _prepare_gated(c, seed):
    g = _generator(seed)
    rows, d = c["rows"], c["d"]
    x = _randn(g, rows, 2 * d)
    x *= 2.0
    return dict(x=x.bfloat16(), q=torch.empty(rows, d, dtype=torch.uint8, device="cuda"),
                scales=torch.empty(rows, _blocks(d), device="cuda"))


def _prepare_quantize(c, seed):
    g = _generator(seed)
    rows, d, r = c["rows"], c["d"], c["block_rows"]
    x = _randn(g, rows, d)
    x = _with_outliers(x, g) if r == 1 else x * 0.02
    return dict(x=x.bfloat16(), q=torch.empty(rows, d, dtype=torch.uint8, device="cuda"),
                scales=torch.empty(-(-rows // r), _blocks(d), device="cuda"))


def _prepare_linear(c, seed):
    g = _generator(seed)
    m, n, k = c["m"], c["n"], c["k"]
    xq, x_scales = _quantised(_with_outliers(_randn(g, m, k), g), 1)
    wq, w_scales = _quantised(_randn(g, n, k) * 0.02, BLOCK)
    return dict(xq=xq.view(torch.uint8), x_scales=x_scales, wq=wq.view(torch.uint8), w_scales=w_scales,
                bias=(0.1 * _randn(g, n)).bfloat16() if c["bias"] else None,
                y=torch.empty(m, n, dtype=torch.bfloat16, device="cuda"))


def prepare(case, seed):
    make = {"norm": _prepare_norm, "gated": _prepare_gated, "quantize": _prepare_quantize, "linear": _prepare_linear}
    return dict(make[case["op"]](case, seed), case=case)


# -------------------------------------------------------------- plain forms

def _in_blocks(y, block_rows):
    """`y` [rows, d] padded with zeros to whole blocks, as [row blocks, block_rows, column blocks, 128]."""
    rows, d = y.shape
    up, across = -(-rows // block_rows), _blocks(d)
    if (up * block_rows, across * BLOCK) != (rows, d):
        y = torch.nn.functional.pad(y, (0, across * BLOCK - d, 0, up * block_rows - rows))
    return y.view(up, block_rows, across, BLOCK)


def _quantised(y, block_rows):
    """E4M3 values of float32 `y` and the scales of its blocks of block_rows x 128."""
    rows, d = y.shape
    b = _in_blocks(y, block_rows)
    scales = (b.abs().amax(3).amax(1) * (1.0 / E4M3_MAX)).clamp(min=LEAST_SCALE)       # [row blocks, column blocks]
    q = (b * (1.0 / scales)[:, None, :, None]).clamp(-E4M3_MAX, E4M3_MAX).to(torch.float8_e4m3fn)
    return q.view(q.shape[0] * block_rows, -1)[:rows, :d].contiguous(), scales


def _spread(scales, rows, cols, block_rows):
    """The scale of every element."""
    s = scales.repeat_interleave(BLOCK, 1)[:, :cols]
    return s if block_rows == 1 else s.repeat_interleave(block_rows, 0)[:rows]


def _act(a, act):
    if act == "gelu_tanh":
        return 0.5 * a * (1.0 + torch.tanh(0.7978845608 * (a + 0.044715 * a * a * a)))
    if act == "gelu_erf":
        return 0.5 * a * (1.0 + torch.erf(a * 0.5 ** 0.5))
    return a / (1.0 + torch.exp(-a)) if act == "silu" else a


def _plain_norm(s):
    r = s["x"].float()
    r = s["res"].float() + (r if s["gate"] is None else s["gate"].float() * r)
    res = r.bfloat16()
    h = res.float()
    y = h * (1.0 / torch.sqrt((h * h).mean(1, keepdim=True) + s["eps"]))
    if s["weight"] is not None:
        y = y * s["weight"].float()
    if s["ada_scale"] is not None:
        y = y * (1.0 + s["ada_scale"].float()) + s["ada_shift"].float()
    q, scales = _quantised(y, 1)
    return {"res": res, "q": q, "scales": scales}


def _plain_gated(s):
    c = s["case"]
    x = s["x"].float()
    q, scales = _quantised(_act(x[:, :c["d"]], c["act"]) * x[:, c["d"]:], 1)
    return {"q": q, "scales": scales}


def _plain_quantize(s):
    q, scales = _quantised(s["x"].float(), s["case"]["block_rows"])
    return {"q": q, "scales": scales}


def _plain_linear(s):
    c = s["case"]
    x = s["xq"].view(torch.float8_e4m3fn).float() * _spread(s["x_scales"], c["m"], c["k"], 1)
    w = s["wq"].view(torch.float8_e4m3fn).float() * _spread(s["w_scales"], c["n"], c["k"], BLOCK)
    a = torch.matmul(x, w.t())
    if s["bias"] is not None:
        a = a + s["bias"].float()
    return {"y": _act(a, c["act"]).bfloat16()}


def _own(s):
    import fusion_add_rmsnorm_gb300 as gbf
    c = s["case"]
    act = {"none": gbf.ACT_NONE, "gelu_tanh": gbf.ACT_GELU_TANH, "gelu_erf": gbf.ACT_GELU_ERF, "silu": gbf.ACT_SILU}
    if c["op"] == "linear":
        gbf.linear_fp8_block(s["xq"], s["x_scales"], s["wq"], s["w_scales"], s["bias"], s["y"], act=act[c["act"]])
        return {"y": s["y"]}
    if c["op"] == "norm":
        mode = {"weight": gbf.NORM_WEIGHT, "noweight": gbf.NORM_NOWEIGHT, "ada": gbf.NORM_ADA}[c["mode"]]
        gbf.add_rmsnorm_fp8_block(s["x"], s["res"], s["res_out"], s["q"], s["scales"], mode, weight=s["weight"],
                                  gate=s["gate"], ada_scale=s["ada_scale"], ada_shift=s["ada_shift"], eps=s["eps"])
    elif c["op"] == "gated":
        gbf.gated_act_fp8_block(s["x"], s["q"], s["scales"], act=act[c["act"]])
    else:
        gbf.quantize_fp8_block(s["x"], s["q"], s["scales"], block_rows=c["block_rows"])
    out = {"q": s["q"].view(torch.float8_e4m3fn), "scales": s["scales"]}
    return dict(out, res=s["res_out"]) if c["op"] == "norm" else out


def run(state):
    if own:
        return _own(state)
    plain = {"norm": _plain_norm, "gated": _plain_gated, "quantize": _plain_quantize, "linear": _plain_linear}
    return plain[state["case"]["op"]](state)


# ------------------------------------------------------------- what it costs

def work(case):
    c = case
    if c["op"] == "linear":
        m, n, k = c["m"], c["n"], c["k"]
        size = m * k + n * k + 4 * _blocks(k) * (m + _blocks(n)) + 2 * m * n + (2 * n if c["bias"] else 0)
        return {"bytes": size, "flops": 2 * m * n * k}
    if c["op"] == "norm":
        cells, vectors = c["rows"] * c["hidden"], {"weight": 1, "noweight": 0, "ada": 2}[c["mode"]] + c["gated"]
        return {"bytes": 7 * cells + 4 * c["rows"] * _blocks(c["hidden"]) + 2 * c["hidden"] * vectors,
                "flops": 8 * cells}
    cells = c["rows"] * c["d"]
    if c["op"] == "gated":
        return {"bytes": 5 * cells + 4 * c["rows"] * _blocks(c["d"]), "flops": 10 * cells}
    return {"bytes": 3 * cells + 4 * -(-c["rows"] // c["block_rows"]) * _blocks(c["d"]), "flops": 3 * cells}


# ----------------------------------------------------------------- in 64 bits

def _exact_codes(y, block_rows):
    """What the codes of float64 `y` stand for before their rounding, and the scales, block column by block column."""
    rows, d = y.shape
    of_row = torch.arange(rows, device=y.device) // block_rows
    codes, scales = torch.empty_like(y), []
    for lo in range(0, d, BLOCK):
        part = y[:, lo:lo + BLOCK]
        top = torch.zeros(int(of_row[-1]) + 1, dtype=torch.float64, device=y.device)
        top.scatter_reduce_(0, of_row, part.abs().amax(1), "amax")
        scale = torch.maximum(top / E4M3_MAX, torch.full_like(top, LEAST_SCALE))
        codes[:, lo:lo + BLOCK] = part / scale[of_row][:, None]
        scales.append(scale)
    return {"q": codes, "scales": torch.stack(scales, 1)}


def _exact_act(a, act):
    if act == "gelu_tanh":
        return a * torch.sigmoid(2 * 0.7978845608 * (a + 0.044715 * a ** 3))
    if act == "gelu_erf":
        return a * 0.5 * torch.erfc(-a / 2 ** 0.5)
    return a * torch.sigmoid(a) if act == "silu" else a


def exact(case, seed):
    c, s = case, prepare(case, seed)
    if c["op"] == "linear":
        y = torch.zeros(c["m"], c["n"], dtype=torch.float64, device="cuda")
        rows = torch.arange(c["n"], device="cuda") // BLOCK
        for j, lo in enumerate(range(0, c["k"], BLOCK)):
            part = s["xq"][:, lo:lo + BLOCK].view(torch.float8_e4m3fn).double() * s["x_scales"][:, j, None].double()
            y.addmm_(part, (s["wq"][:, lo:lo + BLOCK].view(torch.float8_e4m3fn).double()
                            * s["w_scales"][rows, j, None].double()).t())
        if c["bias"]:
            y += s["bias"].double()
        return {"y": _exact_act(y, c["act"])}
    if c["op"] == "norm":
        r = s["x"].double()
        if c["gated"]:
            r *= s["gate"].double()
        r += s["res"].double()
        h = r.float().bfloat16().double()             # the norm reads the residual as it is kept
        y = h * torch.rsqrt(h.square().sum(1) / c["hidden"] + s["eps"])[:, None]
        if c["mode"] == "weight":
            y *= s["weight"].double()
        if c["mode"] == "ada":
            y = torch.addcmul(s["ada_shift"].double(), y, 1 + s["ada_scale"].double())
        return dict(_exact_codes(y, 1), res=r)
    x = s["x"].double()
    if c["op"] == "gated":
        gate, up = x.chunk(2, 1)
        return _exact_codes(_exact_act(gate, c["act"]) * up, 1)
    return _exact_codes(x, c["block_rows"])
