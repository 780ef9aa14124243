"""Workloads of the token operators: the norm of a token stream, 8-bit
quantisation of its rows, and the 8-bit integer matrix product.

A generative model that ends in this framework's waveform decoder carries its
hidden states as a stream [tokens, width]: each block adds its result to the
stream, takes the root-mean-square norm and multiplies by a weight matrix; the
last such product gives the latents that the decoder reads.  Served in 8 bits
a layer is

    h = x + residual,  t = h gain,  q = round(127 t / max|t|),
    scale = max|t| / (127 rms(h)),  y = scale w_scale (q w^T) + bias + residual'

with one scale for each token and one for each channel.  `own = False` runs
the plain form in elementary torch operations, `own = True` the framework's
operators.
"""
import torch

own = False

EPS = 1e-6
DTYPES = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}


def listed():
    return [
        # one token of one listener through a norm: latency alone counts
        {"name": "norm_token", "op": "norm", "dtype": "bf16", "tokens": 1, "width": 4096,
         "residual": True},
        # the frames of a 60 s stereo latent (2400 a side) in the decoder's own type
        {"name": "norm_frames", "op": "norm", "dtype": "f32", "tokens": 4800, "width": 1024,
         "residual": True},
        # a ragged stream whose rows start on odd addresses, without a residual
        {"name": "norm_odd", "op": "norm", "dtype": "f16", "tokens": 2001, "width": 1537,
         "residual": False},
        # the prompts of a whole batch at once
        {"name": "norm_batch", "op": "norm", "dtype": "bf16", "tokens": 16384, "width": 8192,
         "residual": True},
        # one token through norm and projection, as every step of generation does
        {"name": "norm_linear_token", "op": "norm_linear", "dtype": "bf16", "tokens": 1,
         "width": 2048, "channels": 8192, "residual": True, "packed": False},
        # every frame of a minute through norm and projection
        {"name": "norm_linear_frames", "op": "norm_linear", "dtype": "bf16", "tokens": 4800,
         "width": 1024, "channels": 4096, "residual": True, "packed": False},
        # a feed-forward block's second product for a few listeners, added to the stream
        {"name": "linear_few", "op": "linear", "dtype": "f16", "tokens": 24, "width": 8192,
         "channels": 2048, "residual": True, "packed": False},
        # odd sizes, weights stored without padding (rows start on any byte)
        {"name": "linear_odd", "op": "linear", "dtype": "bf16", "tokens": 333, "width": 1111,
         "channels": 777, "residual": False, "packed": True},
        # the projection into the decoder's 32 latent channels, channels first in f32
        {"name": "matmul_latents", "op": "matmul", "dtype": "f32", "tokens": 4800, "width": 1024,
         "channels": 32, "residual": False, "packed": False, "channels_first": True},
        # one token through a square projection: the weights' bytes bound it
        {"name": "matmul_token", "op": "matmul", "dtype": "bf16", "tokens": 1, "width": 4096,
         "channels": 4096, "residual": False, "packed": False, "channels_first": False},
        # ragged in every direction
        {"name": "matmul_ragged", "op": "matmul", "dtype": "f16", "tokens": 1537, "width": 2050,
         "channels": 1111, "residual": True, "packed": False, "channels_first": False},
        # the largest product: a batch of prompts through a wide projection
        {"name": "matmul_batch", "op": "matmul", "dtype": "bf16", "tokens": 8192, "width": 8192,
         "channels": 8192, "residual": False, "packed": False, "channels_first": False},
    ]


def _log_int(rng, lo, hi):
    """Log-uniform whole number in [lo, hi]; half of them rounded to 32."""
    v = int(round(lo * (hi / lo) ** rng.random()))
    if rng.random() < 0.5 and v > 32:
        v = v // 32 * 32
    return max(lo, min(hi, v))


def draw(rng):
    op = rng.choice(("norm", "norm_linear", "linear", "matmul"))
    case = {"op": op, "dtype": rng.choice(("f32", "bf16", "f16")),
            "tokens": _log_int(rng, 1, 16384 if op == "norm" else 8192),
            "width": _log_int(rng, 64, 8192), "residual": rng.random() < 0.5}
    if op == "norm":
        return case
    if op != "matmul" and case["dtype"] == "f32":
        # in f32 a value next to a rounding border of the 8-bit grid decides
        # more than the type's last digits
        case["dtype"] = "bf16"
    case["channels"] = _log_int(rng, 32, 8192)
    case["packed"] = rng.random() < 0.25
    if op == "matmul":
        case["channels_first"] = rng.random() < 0.3
    return case


def _rows_int8(gen, rows, cols, packed):
    """int8 rows as a program keeps them: padded to 16 bytes, or packed."""
    ld = cols if packed else (cols + 15) // 16 * 16
    q = torch.randn((rows, ld), device="cuda", generator=gen).mul_(30).round_().clamp_(-127, 127)
    return q.to(torch.int8)[:, :cols]


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    dt = DTYPES[case["dtype"]]
    m, k = case["tokens"], case["width"]

    def randn(*shape):
        return torch.randn(shape, device="cuda", generator=gen)

    def rand(*shape):
        return torch.rand(shape, device="cuda", generator=gen)

    s = {"case": dict(case)}
    if case["op"] != "matmul":
        # a few channels of a stream are far larger than the others
        loud = 1.0 + 8.0 * (rand(k) > 0.99).float()
        s["x"] = (randn(m, k) * loud).to(dt)
    if case["op"] in ("norm", "norm_linear"):
        s["gain"] = (1.0 + 0.2 * randn(k)).to(dt)
        s["stream"] = (2.0 * randn(m, k) * loud).to(dt) if case["residual"] else None
    if case["op"] != "norm":
        n = case["channels"]
        s["w"] = _rows_int8(gen, n, k, case["packed"])
        s["w_scale"] = 0.0005 + 0.001 * rand(n)
        s["bias"] = 0.1 * randn(n)
    if case["op"] == "matmul":
        s["q"] = _rows_int8(gen, m, k, case["packed"])
        s["scale"] = 0.01 + 0.02 * rand(m)
    if case["op"] in ("linear", "matmul") and case["residual"]:
        n = case["channels"]
        s["skip"] = randn(*((n, m) if case.get("channels_first") else (m, n))).to(dt)
    return s


# ------------------------------------------------------------- the plain form


def _quantise(t):
    """Rows of t as whole numbers in [-127, 127], and max|t| of each."""
    top = t.abs().amax(-1, keepdim=True)
    return (t * (127.0 / top)).round(), top


def _product(q, scale, s, dt):
    """scale w_scale (q w^T) + bias + skip, rounded once to dt."""
    y = (q @ s["w"].float().t()) * scale * s["w_scale"] + s["bias"]
    if s["case"].get("channels_first"):
        y = y.t()
    if s.get("skip") is not None:
        y = y + s["skip"].float()
    return y.to(dt).contiguous()


def _plain(s):
    case = s["case"]
    dt = DTYPES[case["dtype"]]
    if case["op"] == "matmul":
        return {"y": _product(s["q"].float(), s["scale"][:, None], s, dt)}
    h = s["x"].float()
    if case["op"] == "linear":
        q, top = _quantise(h)
        return {"y": _product(q, top / 127.0, s, dt)}
    out = {}
    if s["stream"] is not None:
        h = h + s["stream"].float()
        out["h"] = h.to(dt)
    t = h * s["gain"].float()
    rstd = torch.rsqrt(h.square().mean(-1, keepdim=True) + EPS)
    if case["op"] == "norm":
        out["y"] = (t * rstd).to(dt)
    else:
        q, top = _quantise(t)
        out["y"] = _product(q, top * rstd / 127.0, s, dt)
    return out


# ------------------------------------------------------- the framework's calls


def _own(s):
    from bigvgan_waveform_decoder_alias_b200 import native
    case = s["case"]
    dt = DTYPES[case["dtype"]]
    if case["op"] == "matmul":
        return {"y": native.bv_int8_matmul(s["q"], s["scale"], s["w"], s["w_scale"],
                                           bias=s["bias"], residual=s.get("skip"), out_dtype=dt,
                                           channels_first=case["channels_first"])}
    if case["op"] == "linear":
        q, scale = native.bv_quantize_rows(s["x"])
        return {"y": native.bv_int8_matmul(q, scale, s["w"], s["w_scale"], bias=s["bias"],
                                           residual=s.get("skip"), out_dtype=dt)}
    if case["op"] == "norm":
        if s["stream"] is None:
            return {"y": native.bv_rms_norm(s["x"], s["gain"], eps=EPS)}
        y, h = native.bv_rms_norm(s["x"], s["gain"], eps=EPS, residual=s["stream"])
        return {"y": y, "h": h}
    out = {}
    if s["stream"] is None:
        q, scale = native.bv_rms_norm_int8(s["x"], s["gain"], eps=EPS)
    else:
        q, scale, out["h"] = native.bv_rms_norm_int8(s["x"], s["gain"], eps=EPS,
                                                     residual=s["stream"])
    out["y"] = native.bv_int8_matmul(q, scale, s["w"], s["w_scale"], bias=s["bias"], out_dtype=dt)
    return out


def run(state):
    return _own(state) if own else _plain(state)


# -------------------------------------------------------------- what it takes


def work(case):
    """Bytes: every input read once, every output written once (the 8-bit
    rows between two operators of a pass among them, written and read).
    Operations: two for each product and sum of the matrix product, six for
    each value of a norm, three for each value that is quantised."""
    size = 4 if case["dtype"] == "f32" else 2
    m, k = case["tokens"], case["width"]
    n = case.get("channels", 0)
    nbytes = flops = 0
    if case["op"] in ("norm", "norm_linear"):
        nbytes += m * k * size * (3 if case["residual"] else 1) + k * size
        flops += 6 * m * k
    if case["op"] == "norm":
        nbytes += m * k * size
    if case["op"] == "linear":
        nbytes += m * k * size
    if case["op"] in ("norm_linear", "linear"):
        nbytes += m * k + 4 * m
        flops += 3 * m * k
    if case["op"] != "norm":
        nbytes += m * k + n * k + 4 * m + 8 * n + m * n * size
        flops += 2 * m * n * k
        if case["op"] != "norm_linear" and case["residual"]:
            nbytes += m * n * size
    return {"bytes": nbytes, "flops": flops}


def exact(case, seed):
    """The same outputs from the definitions, in 64 bits."""
    s = prepare(case, seed)
    f = {name: v.double() for name, v in s.items() if isinstance(v, torch.Tensor)}
    out = {}
    if case["op"] == "matmul":
        rows = f["q"] * f["scale"].unsqueeze(1)
    else:
        v, unit = f["x"], 1.0
        if case["op"] != "linear":
            if "stream" in f:
                v = v + f["stream"]
                out["h"] = v
            unit = 1.0 / torch.sqrt(torch.mean(v * v, dim=1, keepdim=True) + EPS)
            v = v * f["gain"]
        if case["op"] == "norm":
            out["y"] = v * unit
            return out
        step = torch.amax(torch.abs(v), dim=1, keepdim=True) / 127.0
        rows = torch.round(v / step) * step * unit
    y = torch.matmul(rows, (f["w"] * f["w_scale"].unsqueeze(1)).T) + f["bias"]
    y = y.T if case.get("channels_first") else y
    out["y"] = (y + f["skip"] if "skip" in f else y).contiguous()
    return out
