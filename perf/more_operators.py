"""Measured cases of the operators around an 8-bit projection: MXFP8
quantisation (and reading back), the projection with bias, activation and
residual in its epilogue, that epilogue's backward, the norm of a residual
stream to which a block's output is added through dropout, forward (into
MXFP8 or the activations' type) and backward, and dropout by itself.

``run`` computes a case either in its plain form (elementary torch operations
in 32 bits, in 64 where a value is rounded to 8 bits afterwards) or, where
``own`` is set, by the library's calls.  An MXFP8 matrix of ``rows`` x ``k`` is
a pair of byte tensors: ``data`` [rows, 32*ceil(k/32)] of E4M3 codes and
``scales``, one E8M0 byte per 32 elements in tiles of 128 rows x 4 blocks (row
r, block j of a tile at (r % 32) * 16 + (r // 32) * 4 + j).  What is held in 8
bits is returned as bfloat16 values, which hold it exactly.
"""
import math

import torch

own = False

DTYPES = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}
SIZE = {"f32": 4, "bf16": 2, "f16": 2}
EPS = 1e-6
ACTS = ("none", "relu", "silu", "gelu", "gelu_tanh")


def listed():
    return [
        # The last, ragged micro-batch of bf16 activations, odd in both sizes, for the forward and the weight gradient's product.
        dict(name="quantize_ragged", op="quantize", rows=777, cols=2061, dtype="bf16", dirs="both", scale="ceil"),
        # The master weights of an MLP projection after an optimiser step, for the forward and the input gradient's product.
        dict(name="quantize_weight", op="quantize", rows=14336, cols=4096, dtype="f32", dirs="both", scale="floor"),
        # One token through the MLP's last projection, added to the residual stream while serving: the weights' bytes alone.
        dict(name="linear_token", op="linear", m=1, n=4096, k=14336, out="bf16", act="none", bias=True, pre=False, res=True),
        # A training batch through the MLP's first projection; the values before the activation are kept for the backward pass.
        dict(name="linear_batch", op="linear", m=16384, n=14336, k=4096, out="bf16", act="gelu_tanh", bias=True, pre=True, res=False),
        # The gradient through an activation of odd sizes, in the activations' type, with the bias's.
        dict(name="act_bwd_ragged", op="act_bwd", rows=777, cols=2061, dtype="f16", act="silu", dz=True, bias=True, dirs="none"),
        # The gradient through the MLP's activation over a training batch, in 8 bits for both gradient products, with the bias's.
        dict(name="act_bwd_batch", op="act_bwd", rows=16384, cols=14336, dtype="bf16", act="gelu_tanh", dz=False, bias=True, dirs="both"),
        # One token between two blocks while serving, into the 8 bits that the next projection takes.
        dict(name="norm_fwd_token", op="norm_fwd", rows=1, cols=4096, dtype="bf16", x=True, p=0.0, to="q"),
        # A training batch between two blocks with dropout on the branch, into 8 bits.
        dict(name="norm_fwd_batch", op="norm_fwd", rows=16384, cols=4096, dtype="bf16", x=True, p=0.1, to="q"),
        # The backward of a ragged fp32 batch.
        dict(name="norm_bwd_ragged", op="norm_bwd", rows=1001, cols=1111, dtype="f32", x=True, p=0.1),
        # The backward of the training batch.
        dict(name="norm_bwd_batch", op="norm_bwd", rows=16384, cols=4096, dtype="bf16", x=True, p=0.1),
        # Dropout of a small model's embeddings, odd in both sizes.
        dict(name="dropout_ragged", op="dropout", rows=777, cols=2061, dtype="f32", p=0.1, res=False),
        # Dropout of a training batch's hidden activations, added to what passes by them.
        dict(name="dropout_batch", op="dropout", rows=16384, cols=14336, dtype="bf16", p=0.1, res=True),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["quantize", "linear", "act_bwd", "norm_fwd", "norm_bwd", "dropout"])
    dtype = rng.choice(["f32", "bf16", "f16"])
    if op == "linear":
        n, k = _log(rng, 100, 16384), _log(rng, 64, 16384)
        return dict(op=op, m=_log(rng, 1, min(16384, (1 << 39) // (n * k), (1 << 27) // n)), n=n, k=k, out=dtype, act=rng.choice(ACTS),
                    bias=rng.random() < 0.7, pre=rng.random() < 0.5, res=rng.random() < 0.5)
    cols = _log(rng, 33, 16384)
    rows = _log(rng, 1, min(65536, (1 << 26) // cols))
    if op == "quantize":
        return dict(op=op, rows=rows, cols=cols, dtype=dtype, dirs=rng.choice(["rows", "cols", "both"]), scale=rng.choice(["floor", "ceil"]))
    if op == "act_bwd":
        dirs = rng.choice(["none", "rows", "both"])
        return dict(op=op, rows=rows, cols=cols, dtype=dtype, act=rng.choice(ACTS), dz=dirs == "none" or rng.random() < 0.5,
                    bias=rng.random() < 0.7, dirs=dirs)
    p = rng.choice([0.0, 0.1, 0.5])
    if op == "dropout":
        return dict(op=op, rows=rows, cols=cols, dtype=dtype, p=p, res=rng.random() < 0.5)
    rows = min(rows, (1 << 25) // cols)
    case = dict(op=op, rows=rows, cols=cols, dtype=dtype, x=rng.random() < 0.8, p=p)
    if op == "norm_fwd":
        case["to"] = rng.choice(["q", "h", "both"])
    return case


def _blocks(k):
    return -(-k // 32)


def _mx_bytes(rows, k):
    return rows * _blocks(k) * 33


def work(case):
    op = case["op"]
    if op == "linear":
        m, n, k, s = case["m"], case["n"], case["k"], SIZE[case["out"]]
        return {"bytes": _mx_bytes(m, k) + _mx_bytes(n, k) + m * n * s * (1 + case["pre"] + case["res"]) + (4 * n if case["bias"] else 0),
                "flops": 2 * m * n * k}
    rows, cols, s = case["rows"], case["cols"], SIZE[case["dtype"]]
    n = rows * cols

    def packed(dirs):  # written, read back, and the values written
        return sum(2 * _mx_bytes(*d) + 2 * n for d in ([(rows, cols)] if dirs in ("rows", "both") else []) +
                   ([(cols, rows)] if dirs in ("cols", "both") else []))
    if op == "quantize":
        return {"bytes": n * s + packed(case["dirs"]), "flops": 0}
    if op == "act_bwd":
        reads = 1 if case["act"] == "none" else 2
        return {"bytes": n * s * (reads + case["dz"]) + packed(case["dirs"]) + (4 * cols if case["bias"] else 0), "flops": 12 * n}
    if op == "dropout":
        return {"bytes": n * s * (2 + case["res"]), "flops": 2 * n}
    if op == "norm_fwd":
        to = case["to"]
        return {"bytes": n * s * (2 + case["x"] + (to != "q")) + (packed("rows") if to != "h" else 0) + 4 * cols + 4 * rows, "flops": 6 * n}
    return {"bytes": n * s * (4 + (case["x"] and case["p"] > 0)) + 8 * cols + 4 * rows, "flops": 12 * n}


# ------------------------------------------------------------ plain MXFP8

def _pow2(e):
    """2^e in fp32, from its bits: e in [-127, 127], -127 being subnormal."""
    e = e.to(torch.int32)
    return torch.where(e > -127, (e + 127) << 23, torch.full_like(e, 1 << 22)).view(torch.float32)


def _split(x, scale):
    """Values on the E4M3 grid and block exponents of the rows of x (fp32 or fp64), in blocks of 32, zero padded."""
    rows, k = x.shape
    x = torch.nn.functional.pad(x, (0, _blocks(k) * 32 - k)).view(rows, -1, 32)
    amax = x.abs().amax(-1)
    mant, e = torch.frexp(amax)  # amax = mant 2^e, mant in [1/2, 1)
    e = e - 9
    if scale == "ceil":
        e = e + (mant > 0.875).to(e.dtype)  # 448 = 0.875 * 2^9
    e = torch.where(amax > 0, e, torch.full_like(e, -127)).clamp(-127, 127)
    v = (x.abs() / _pow2(e).to(x.dtype).unsqueeze(-1)).clamp(max=448.0)
    ve = torch.frexp(v)[1] - 1  # v in [2^ve, 2 * 2^ve); 2^-6 and below share a step
    step = _pow2(ve.clamp(min=-6) - 3).to(x.dtype)
    return torch.copysign(torch.round(v / step) * step, x), e


def _values(x, scale):
    q, e = _split(x, scale)
    return (q * _pow2(e).to(q.dtype).unsqueeze(-1)).view(x.shape[0], -1)[:, : x.shape[1]].to(torch.bfloat16)


def _pack(x):
    """An MXFP8 matrix (floor scales) of the rows of x, laid out as the library takes it."""
    q, e = _split(x, "floor")
    rows, nb = e.shape
    mag = q.abs()
    ve = (torch.frexp(mag)[1] - 1).clamp(min=-6)
    man = (mag / _pow2(ve - 3)).to(torch.int32)  # 8 + mantissa, below 8 for subnormals
    code = torch.where(mag >= 2.0 ** -6, (ve + 6) * 8 + man, man)
    code = (code + 128 * torch.signbit(q).to(torch.int32)).to(torch.uint8).view(rows, nb * 32)
    rt, kt = -(-rows // 128), -(-nb // 4)
    s = torch.nn.functional.pad((e + 127).to(torch.uint8), (0, kt * 4 - nb, 0, rt * 128 - rows))
    return code.contiguous(), s.view(rt, 4, 32, kt, 4).permute(0, 3, 2, 1, 4).reshape(-1).contiguous()


def _unpack(q, rows, k):
    data, scales = q
    nb = _blocks(k)
    rt, kt = -(-rows // 128), -(-nb // 4)
    code = torch.arange(256, device=data.device)
    mag = torch.where((code & 120) > 0, (8 + (code & 7)) * 2.0 ** ((code >> 3 & 15) - 10).float(), (code & 7) * 2.0 ** -9)
    grid = torch.where(code >= 128, -mag, mag)
    v = grid[data.to(torch.int32)].view(rows, nb, 32)
    e = scales.view(rt, kt, 32, 4, 4).permute(0, 3, 2, 1, 4).reshape(rt * 128, kt * 4)[:rows, :nb].to(torch.int32) - 127
    return (v * _pow2(e).unsqueeze(-1)).view(rows, nb * 32)[:, :k]


def _mx_empty(rows, k):
    tiles = (-(-rows // 128)) * (-(-_blocks(k) // 4))
    return (torch.empty((rows, _blocks(k) * 32), dtype=torch.uint8, device="cuda"),
            torch.empty(tiles * 512, dtype=torch.uint8, device="cuda"))


# ------------------------------------------------------------ plain dropout

def _keep(rows, cols, p, seed, offset):
    """Which elements stay: 16 bits each of Philox4x32-10 of key ``seed`` and
    counter (column / 8, row, offset), at least round(65536 p)."""
    groups = -(-cols // 8)
    low = 0xFFFFFFFF
    at = torch.arange(rows * groups, device="cuda", dtype=torch.int64)
    c = [at % groups, at // groups, torch.full_like(at, offset & low), torch.full_like(at, offset >> 32)]
    k0, k1 = seed & low, seed >> 32
    for _ in range(10):
        a, b = c[0] * 0xD2511F53, c[2] * 0xCD9E8D57  # modulo 2^64
        c = [(b >> 32 & low) ^ c[1] ^ k0, b & low, (a >> 32 & low) ^ c[3] ^ k1, a & low]
        k0, k1 = (k0 + 0x9E3779B9) & low, (k1 + 0xBB67AE85) & low
    words = torch.stack(c, -1)
    bits = torch.stack((words & 0xFFFF, words >> 16), -1).view(rows, groups * 8)[:, :cols]
    return bits >= _threshold(p)


def _threshold(p):
    return int(math.floor(p * 65536 + 0.5))


def _drop(v, s):
    """v through the state's dropout, in v's type."""
    case = s["case"]
    if case["p"] == 0:
        return v
    t = _threshold(case["p"])
    return torch.where(_keep(case["rows"], case["cols"], case["p"], s["seed"], s["offset"]), v * (65536 / (65536 - t)), torch.zeros_like(v))


# ------------------------------------------------------------ inputs

def _activations(shape, g, dtype, spread=1.0):
    """Normal values whose rows and columns differ in size, as activations and gradients do."""
    t = torch.randn(shape, generator=g, device="cuda", dtype=torch.float32)
    t *= torch.exp(0.5 * spread * torch.randn((shape[0], 1), generator=g, device="cuda"))
    t *= torch.exp(0.5 * spread * torch.randn((1, shape[1]), generator=g, device="cuda"))
    return t.to(dtype)


def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(int(seed))
    s = {"case": case, "seed": (int(seed) * 0x9E3779B97F4A7C15 + 12345) & 0xFFFFFFFFFFFFFFFF, "offset": 7 + (int(seed) % 1000 << 33)}
    op = case["op"]
    if op == "linear":
        m, n, k, dt = case["m"], case["n"], case["k"], DTYPES[case["out"]]
        s["a"] = _pack(_activations((m, k), g, torch.float32))
        s["b"] = _pack(torch.randn((n, k), generator=g, device="cuda") / math.sqrt(k))
        s["bias"] = 0.2 * torch.randn(n, generator=g, device="cuda") if case["bias"] else None
        s["res"] = torch.randn((m, n), generator=g, device="cuda").to(dt) if case["res"] else None
        s["pre"] = torch.empty((m, n), dtype=dt, device="cuda") if case["pre"] else None
        s["out"] = torch.empty((m, n), dtype=dt, device="cuda")
        return s
    rows, cols, dt = case["rows"], case["cols"], DTYPES[case["dtype"]]

    def like(dtype=dt):
        return torch.empty((rows, cols), dtype=dtype, device="cuda")

    def packed(dirs):
        r, c = dirs in ("rows", "both"), dirs in ("cols", "both")
        s["by_rows"], s["by_cols"] = _mx_empty(rows, cols) if r else None, _mx_empty(cols, rows) if c else None
        s["rows_out"] = like(torch.bfloat16) if r else None
        s["cols_out"] = torch.empty((cols, rows), dtype=torch.bfloat16, device="cuda") if c else None
    if op == "quantize":
        s["x"] = _activations((rows, cols), g, dt)
        packed(case["dirs"])
        return s
    if op == "act_bwd":
        s["dout"] = _activations((rows, cols), g, dt, 0.5)
        s["pre"] = None if case["act"] == "none" else _activations((rows, cols), g, dt, 0.5)
        s["dz"] = like() if case["dz"] else None
        s["d_bias"] = torch.empty(cols, device="cuda") if case["bias"] else None
        packed(case["dirs"])
        return s
    if op == "dropout":
        s["x"] = _activations((rows, cols), g, dt, 0.5)
        s["res"] = _activations((rows, cols), g, dt, 0.5) if case["res"] else None
        s["out"] = like()
        return s
    s["x"] = _activations((rows, cols), g, dt, 0.5) if case["x"] else None
    s["f"] = _activations((rows, cols), g, dt, 0.5)
    s["w"] = 1 + 0.2 * torch.randn(cols, generator=g, device="cuda")
    if op == "norm_fwd":
        s["y"], s["h"] = like(), like() if case["to"] != "q" else None
        s["rstd"] = torch.empty(rows, device="cuda")
        packed("rows" if case["to"] != "h" else "none")
        return s
    s["y"], _, s["rstd"] = _norm_fwd(s, torch.float32)
    s["dy"] = _activations((rows, cols), g, dt, 0.5)
    s["dh"] = _activations((rows, cols), g, dt, 0.5)
    s["x"] = s["f"] = None
    s["df"] = like()
    s["dx"] = like() if case["x"] and case["p"] > 0 else None  # without dropout both gradients are the same
    s["d_w"] = torch.empty(cols, device="cuda")
    return s


# ------------------------------------------------------------ plain operators

def _norm_fwd(s, wide):
    """y in the activations' type, h in ``wide``, 1 / rms."""
    y = _drop(s["f"].to(wide), s)
    if s["x"] is not None:
        y = y + s["x"].to(wide)
    r = torch.rsqrt((y * y).mean(-1, keepdim=True) + EPS)
    return y.to(s["f"].dtype), y * r * s["w"], r[:, 0].to(torch.float32)


def _norm_bwd(s):
    dt = s["y"].dtype
    y, dy, dh = s["y"].to(torch.float32), s["dy"].to(torch.float32), s["dh"].to(torch.float32)
    r = s["rstd"].unsqueeze(1)
    yn, g = y * r, dh * s["w"]
    t = dy + r * (g - yn * (g * yn).mean(-1, keepdim=True))
    return {"dx": None if s["dx"] is None else t.to(dt), "df": _drop(t, s).to(dt), "d_w": (dh * yn).sum(0)}


def _act(z, act):
    if act == "relu":
        return torch.where(z > 0, z, torch.zeros_like(z))
    if act == "silu":
        return z / (1 + torch.exp(-z))
    if act == "gelu":
        return 0.5 * z * torch.erfc(-z * math.sqrt(0.5))
    if act == "gelu_tanh":  # 1 + tanh(u) = 2 / (1 + exp(-2u))
        return z / (1 + torch.exp(-2 * math.sqrt(2 / math.pi) * (z + 0.044715 * z * z * z)))
    return z


def _act_slope(z, act):
    if act == "relu":
        return (z > 0).to(z.dtype)
    if act == "silu":
        sig = 1 / (1 + torch.exp(-z))
        return sig * (1 + z * (1 - sig))
    if act == "gelu":
        return 0.5 * torch.erfc(-z * math.sqrt(0.5)) + z * torch.exp(-0.5 * z * z) / math.sqrt(2 * math.pi)
    c = 2 * math.sqrt(2 / math.pi)
    sig = 1 / (1 + torch.exp(-c * (z + 0.044715 * z * z * z)))
    return sig * (1 + z * (1 - sig) * c * (1 + 3 * 0.044715 * z * z))


# ------------------------------------------------------------ run

_kept = {}


def _handle():
    if "h" not in _kept:
        import newton_schulz_nesterov_gb300 as dm
        _kept["dm"], _kept["h"] = dm, dm.Handle(0)
    return _kept["h"]


def _read_back(s, h):
    if s["by_rows"] is not None:
        h.mxfp8_dequantize(s["by_rows"], s["rows_out"])
    if s["by_cols"] is not None:
        h.mxfp8_dequantize(s["by_cols"], s["cols_out"])
    return {"rows": s["rows_out"], "cols": s["cols_out"]}


def _run_own(s):
    h, case = _handle(), s["case"]
    op = case["op"]
    if op == "quantize":
        h.mxfp8_quantize(s["x"], s["by_rows"], s["by_cols"], scale=case["scale"])
        return _read_back(s, h)
    if op == "linear":
        h.mx_linear(s["a"], s["b"], s["out"], case["k"], bias=s["bias"], act=case["act"], pre=s["pre"], residual=s["res"])
        return {"out": s["out"], "pre": s["pre"]}
    if op == "act_bwd":
        h.act_backward(s["dout"], s["pre"], case["act"], dz=s["dz"], d_bias=s["d_bias"], by_rows=s["by_rows"], by_cols=s["by_cols"])
        return dict(_read_back(s, h), dz=s["dz"], d_bias=s["d_bias"])
    if op == "dropout":
        h.dropout(s["x"], s["out"], case["p"], s["seed"], s["offset"], residual=s["res"])
        return s["out"]
    if op == "norm_fwd":
        h.add_norm_forward(s["x"], s["f"], s["w"], s["y"], s["rstd"], out=s["h"], q=s["by_rows"], p=case["p"], seed=s["seed"],
                           offset=s["offset"], eps=EPS)
        return dict(_read_back(s, h), y=s["y"], h=s["h"], rstd=s["rstd"])
    h.add_norm_backward(s["dy"], s["dh"], s["y"], s["w"], s["rstd"], s["dx"], s["df"], s["d_w"], p=case["p"], seed=s["seed"],
                        offset=s["offset"])
    return {k: s[k] for k in ("dx", "df", "d_w")}


def run(s):
    if own:
        return _run_own(s)
    case = s["case"]
    op = case["op"]
    if op == "quantize":
        x = s["x"].to(torch.float32)
        return {"rows": None if s["by_rows"] is None else _values(x, case["scale"]),
                "cols": None if s["by_cols"] is None else _values(x.t(), case["scale"])}
    if op == "linear":
        z = _unpack(s["a"], case["m"], case["k"]) @ _unpack(s["b"], case["n"], case["k"]).t()
        if s["bias"] is not None:
            z = z + s["bias"]
        out = _act(z, case["act"])
        if s["res"] is not None:
            out = out + s["res"].to(torch.float32)
        dt = s["out"].dtype
        return {"out": out.to(dt), "pre": z.to(dt) if case["pre"] else None}
    if op == "act_bwd":
        dz = s["dout"].to(torch.float32)
        if case["act"] != "none":
            dz = dz * _act_slope(s["pre"].to(torch.float32), case["act"])
        return {"rows": None if s["by_rows"] is None else _values(dz, "floor"), "cols": None if s["by_cols"] is None else _values(dz.t(), "floor"),
                "dz": dz.to(s["dout"].dtype) if case["dz"] else None, "d_bias": dz.sum(0) if case["bias"] else None}
    if op == "dropout":
        v = _drop(s["x"].to(torch.float32), s)
        return (v if s["res"] is None else v + s["res"].to(torch.float32)).to(s["out"].dtype)
    if op == "norm_fwd":
        y, h, r = _norm_fwd(s, torch.float64 if case["to"] != "h" else torch.float32)
        return {"rows": _values(h, "floor") if case["to"] != "h" else None, "cols": None, "y": y,
                "h": h.to(y.dtype) if case["to"] != "q" else None, "rstd": r}
    return _norm_bwd(s)


# ------------------------------------------------------------ 64 bits

def exact(case, seed):
    s = prepare(case, seed)
    dev, f64 = "cuda", torch.float64
    op = case["op"]

    def two_to(e):
        return ((e.to(torch.int64) + 1023) << 52).view(f64)

    def positive():
        """The E4M3 values from 0 to 448."""
        code = torch.arange(127, device=dev)
        return torch.where(code < 8, code.to(f64) / 512, (1 + (code % 8).to(f64) / 8) * two_to(code // 8 - 7))

    def read_back(x, scale="floor"):
        """Rows of x quantised and read back, by looking its values up between the grid's midpoints."""
        rows, k = x.shape
        wide = -(-k // 32) * 32
        grid = positive()
        middle = (grid[1:] + grid[:-1]) / 2
        out = torch.empty((rows, k), dtype=f64, device=dev)
        per = max(1, (1 << 25) // wide)
        for i in range(0, rows, per):
            part = x[i:i + per].to(f64)
            full = torch.zeros((part.shape[0], wide), dtype=f64, device=dev)
            full[:, :k] = part
            b = full.view(part.shape[0], -1, 32)
            top = b.abs().amax(-1, keepdim=True)
            safe = torch.where(top > 0, top, torch.ones_like(top))
            if scale == "floor":  # 256 * 2^e <= top < 512 * 2^e
                e = torch.floor(torch.log2(safe)) - 8
                e = e + (safe >= 512 * two_to(e)).to(f64) - (safe < 256 * two_to(e)).to(f64)
            else:  # 224 * 2^e < top <= 448 * 2^e
                e = torch.ceil(torch.log2(safe / 448))
                e = e + (safe > 448 * two_to(e)).to(f64) - (safe <= 224 * two_to(e)).to(f64)
            unit = two_to(torch.where(top > 0, e, torch.full_like(e, -127)).clamp(-127, 127))
            v = b.abs() / unit
            lo = torch.bucketize(v, middle)  # a tie goes below here ...
            tie = (v == middle[lo.clamp(max=125)]) & (lo < 126)
            lo = lo + (tie & (lo % 2 == 1)).to(lo.dtype)  # ... and to the even code
            out[i:i + per] = (torch.copysign(grid[lo], b) * unit).view(part.shape[0], -1)[:, :k]
        return out

    def decoded(q, rows, k):
        """An MXFP8 matrix in 64 bits, from the bits of its codes."""
        code = q[0].to(torch.int32)
        exp, man = (code // 8) % 16, (code % 8).to(f64)
        mag = torch.where(exp == 0, man / 512, (1 + man / 8) * two_to(exp - 7))
        r, j = torch.arange(rows, device=dev)[:, None], torch.arange(q[0].shape[1] // 32, device=dev)[None, :]
        at = ((r // 128) * (-(-q[0].shape[1] // 128)) + j // 4) * 512 + (r % 32) * 16 + (r % 128) // 32 * 4 + j % 4
        unit = two_to(q[1][at].to(torch.int64) - 127)
        return (torch.where(code >= 128, -mag, mag).view(rows, -1, 32) * unit[:, :, None]).view(rows, -1)[:, :k]

    def factors():
        """0 or 1 / (1 - p) of every element: the generator's rounds on 16-bit halves."""
        rows, cols, p = case["rows"], case["cols"], case["p"]
        cut = math.floor(p * 65536 + 0.5)
        if cut == 0:
            return 1.0
        out = torch.empty((rows, cols), dtype=f64, device=dev)
        n = (cols + 7) // 8
        per = max(1, (1 << 22) // n)

        def times(v, c):  # low and high words of the product
            small, big = (v & 65535) * c, (v >> 16) * c
            total = big + (small >> 16)
            return ((total & 65535) << 16) | (small & 65535), total >> 16
        for i in range(0, rows, per):
            m = min(per, rows - i)
            x0 = torch.arange(n, device=dev).repeat(m)
            x1 = torch.arange(i, i + m, device=dev).repeat_interleave(n)
            x2 = torch.full_like(x0, s["offset"] % 2 ** 32)
            x3 = torch.full_like(x0, s["offset"] // 2 ** 32)
            for j in range(10):
                k0 = (s["seed"] % 2 ** 32 + j * 0x9E3779B9) % 2 ** 32
                k1 = (s["seed"] // 2 ** 32 + j * 0xBB67AE85) % 2 ** 32
                l0, h0 = times(x0, 0xD2511F53)
                l1, h1 = times(x2, 0xCD9E8D57)
                x0, x1, x2, x3 = h1 ^ x1 ^ k0, l1, h0 ^ x3 ^ k1, l0
            for j, word in enumerate((x0, x1, x2, x3)):
                for half in range(2):
                    c = 2 * j + half
                    take = (cols - c + 7) // 8
                    if take > 0:
                        bits = (word // 65536 if half else word % 65536).view(m, n)[:, :take]
                        out[i:i + m, c::8] = (bits >= cut).to(f64) * (65536 / (65536 - cut))
        return out

    def normal_below(z):
        return 0.5 * torch.special.erfc(-z / math.sqrt(2))

    if op == "quantize":
        return {"rows": read_back(s["x"], case["scale"]) if s["by_rows"] is not None else None,
                "cols": read_back(s["x"].t(), case["scale"]) if s["by_cols"] is not None else None}
    if op == "linear":
        z = decoded(s["a"], case["m"], case["k"]) @ decoded(s["b"], case["n"], case["k"]).t()
        if s["bias"] is not None:
            z += s["bias"].to(f64)
        act = case["act"]
        if act == "relu":
            out = z.clamp(min=0)
        elif act == "silu":
            out = z * torch.sigmoid(z)
        elif act == "gelu":
            out = z * normal_below(z)
        elif act == "gelu_tanh":
            out = z * torch.sigmoid(math.sqrt(8 / math.pi) * (z + 0.044715 * z ** 3))
        else:
            out = z
        if s["res"] is not None:
            out = out + s["res"].to(f64)
        return {"out": out, "pre": z if case["pre"] else None}
    if op == "act_bwd":
        dz, act = s["dout"].to(f64), case["act"]
        if act != "none":
            z = s["pre"].to(f64)
            if act == "relu":
                dz = dz * (z > 0)
            elif act == "silu":
                dz = dz * (torch.sigmoid(z) + z * torch.sigmoid(z) * torch.sigmoid(-z))
            elif act == "gelu":
                dz = dz * (normal_below(z) + z * torch.exp(-z * z / 2) / math.sqrt(2 * math.pi))
            else:
                u, du = math.sqrt(8 / math.pi) * (z + 0.044715 * z ** 3), math.sqrt(8 / math.pi) * (1 + 0.134145 * z * z)
                dz = dz * (torch.sigmoid(u) + z * du * torch.sigmoid(u) * torch.sigmoid(-u))
        return {"rows": read_back(dz) if s["by_rows"] is not None else None, "cols": read_back(dz.t()) if s["by_cols"] is not None else None,
                "dz": dz if case["dz"] else None, "d_bias": dz.sum(0) if case["bias"] else None}
    if op == "dropout":
        out = s["x"].to(f64) * factors()
        return out if s["res"] is None else out + s["res"].to(f64)
    cols, w = case["cols"], s["w"].to(f64)
    if op == "norm_fwd":
        y = s["f"].to(f64) * factors()
        if s["x"] is not None:
            y = y + s["x"].to(f64)
        r = (y.square().sum(-1) / cols + EPS) ** -0.5
        h = w * (y * r[:, None])
        return {"rows": read_back(h) if case["to"] != "h" else None, "cols": None, "y": y, "h": h if case["to"] != "q" else None, "rstd": r}
    y, dy, dh, r = s["y"].to(f64), s["dy"].to(f64), s["dh"].to(f64), s["rstd"].to(f64)[:, None]
    into = dh * w * r
    t = dy + into - y * (into * y).sum(-1, keepdim=True) * r ** 2 / cols
    return {"dx": None if s["dx"] is None else t, "df": t * factors(), "d_w": (dh * y * r).sum(0)}
