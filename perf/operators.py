"""Measured cases of the operators around a 4-bit projection: MXFP4
quantisation (and reading back), the MXFP4 product, and the norms after and
before a block with its gate and residual scale, forward and backward.

``run`` computes a case either in its plain form (elementary torch operations
in 32 bits) or, where ``own`` is set, by the library's calls.  An MXFP4 matrix
of ``rows`` x ``k`` is a pair of byte tensors: ``data`` [rows, 16*ceil(k/32)],
two elements a byte with the even one in the low half, and ``scales``, one
E8M0 byte per 32 elements in tiles of 128 rows x 4 blocks (row r, block j of a
tile at (r % 32) * 16 + (r // 32) * 4 + j).
"""
import math

import torch

own = False

DTYPES = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}
SIZE = {"f32": 4, "bf16": 2, "f16": 2}
EPS = 1e-6


def listed():
    return [
        # One token's activations before a projection while serving: latency alone.
        dict(name="quantize_token", op="quantize", rows=1, cols=4096, dtype="bf16", dirs="rows", scale="floor", noise=False),
        # A last, ragged micro-batch of fp32 gradients, odd in both sizes, both directions, stochastic rounding.
        dict(name="quantize_ragged", op="quantize", rows=777, cols=2061, dtype="f32", dirs="both", scale="ceil", noise=True),
        # The master weights of an MLP projection after an optimiser step, for the forward and the input-gradient product.
        dict(name="quantize_weight", op="quantize", rows=14336, cols=4096, dtype="f32", dirs="both", scale="floor", noise=False),
        # Output gradients of the same projection over a training batch, for both gradient products.
        dict(name="quantize_grad", op="quantize", rows=16384, cols=14336, dtype="bf16", dirs="both", scale="ceil", noise=True),
        # One token through an MLP projection while serving: the weights' bytes alone.
        dict(name="gemm_token", op="gemm", m=1, n=14336, k=4096, out="bf16", beta=0.0),
        # A short prompt through odd sizes.
        dict(name="gemm_ragged", op="gemm", m=77, n=1111, k=2061, out="f16", beta=0.0),
        # The weight gradient of an MLP projection, added to the fp32 gradient that the optimiser step takes.
        dict(name="gemm_wgrad", op="gemm", m=14336, n=4096, k=8192, out="f32", beta=1.0),
        # A training batch through an MLP projection.
        dict(name="gemm_batch", op="gemm", m=16384, n=14336, k=4096, out="bf16", beta=0.0),
        # One token between two blocks while serving.
        dict(name="norm_fwd_token", op="norm_fwd", rows=1, cols=4096, dtype="bf16", per_gate=1, gate=True, res=False),
        # A training batch between two blocks, a gate per sequence.
        dict(name="norm_fwd_batch", op="norm_fwd", rows=16384, cols=4096, dtype="bf16", per_gate=2048, gate=True, res=True),
        # The backward of a ragged fp32 batch with groups of odd length.
        dict(name="norm_bwd_ragged", op="norm_bwd", rows=1001, cols=1111, dtype="f32", per_gate=77, gate=True, res=True),
        # The backward of the training batch.
        dict(name="norm_bwd_batch", op="norm_bwd", rows=16384, cols=4096, dtype="bf16", per_gate=2048, gate=True, res=True),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["quantize", "gemm", "norm_fwd", "norm_bwd"])
    if op == "quantize":
        cols = _log(rng, 33, 16384)
        return dict(op=op, rows=_log(rng, 1, min(32768, (1 << 26) // cols)), cols=cols, dtype=rng.choice(["f32", "bf16", "f16"]),
                    dirs=rng.choice(["rows", "cols", "both"]), scale=rng.choice(["floor", "ceil"]), noise=rng.random() < 0.5)
    if op == "gemm":
        n, k = _log(rng, 100, 16384), _log(rng, 64, 16384)
        return dict(op=op, m=_log(rng, 1, min(16384, (1 << 39) // (n * k), (1 << 27) // n)), n=n, k=k, out=rng.choice(["f32", "bf16", "f16"]),
                    beta=rng.choice([0.0, 1.0]))
    cols = _log(rng, 64, 16384)
    rows = _log(rng, 1, min(65536, (1 << 25) // cols))
    gate = rng.random() < 0.7
    # A gate row per 16 rows or more: fewer would make the gate a second activation.
    return dict(op=op, rows=rows, cols=cols, dtype=rng.choice(["f32", "bf16", "f16"]),
                per_gate=_log(rng, min(16, rows), rows) if gate else rows, gate=gate, res=rng.random() < 0.5)


def _blocks(k):
    return -(-k // 32)


def _mx_bytes(rows, k):
    return rows * _blocks(k) * 17


def work(case):
    if case["op"] == "quantize":
        n, s = case["rows"] * case["cols"], SIZE[case["dtype"]]
        b = n * s + (n if case["noise"] else 0)
        # packed bytes written, read back, and the values written
        b += (2 * _mx_bytes(case["rows"], case["cols"]) + n * s) if case["dirs"] in ("rows", "both") else 0
        b += (2 * _mx_bytes(case["cols"], case["rows"]) + n * s) if case["dirs"] in ("cols", "both") else 0
        return {"bytes": b, "flops": 0}
    if case["op"] == "gemm":
        m, n, k = case["m"], case["n"], case["k"]
        return {"bytes": _mx_bytes(m, k) + _mx_bytes(n, k) + m * n * SIZE[case["out"]] * (2 if case["beta"] else 1),
                "flops": 2 * m * n * k}
    n, s = case["rows"] * case["cols"], SIZE[case["dtype"]]
    cols, groups = case["cols"], -(-case["rows"] // case["per_gate"]) if case["gate"] else 0
    small = 4 * cols * (2 + groups + (1 if case["res"] else 0)) + 8 * case["rows"]
    if case["op"] == "norm_fwd":
        return {"bytes": 4 * n * s + small, "flops": 10 * n}
    return {"bytes": (7 if case["res"] else 6) * n * s + 2 * small, "flops": 25 * n}


# ------------------------------------------------------------ plain MXFP4

def _pow2(e):
    """2^e in fp32, from its bits: e in [-127, 127], -127 being subnormal."""
    e = e.to(torch.int32)
    return torch.where(e > -127, (e + 127) << 23, torch.full_like(e, 1 << 22)).view(torch.float32)


def _exponent(amax, scale):
    """Block exponent from the block's largest magnitude (fp32)."""
    mant, e = torch.frexp(amax)  # amax = mant 2^e, mant in [1/2, 1)
    e = e - 3
    if scale == "ceil":
        e = e + (mant > 0.75).to(e.dtype)
    return torch.where(amax > 0, e, torch.full_like(e, -127)).clamp(-127, 127)


def _round(v, noise):
    """|x| / 2^e on the E2M1 grid {0, 1/2, 1, 3/2, 2, 3, 4, 6}."""
    v = v.clamp(max=6.0)
    step = torch.where(v < 2, 0.5, torch.where(v < 4, 1.0, 2.0))
    if noise is None:
        return torch.round(v / step) * step
    lo = torch.floor(v / step)
    up = ((v / step - lo) * 256 > noise.to(torch.float32) + 0.5).to(torch.float32)
    return (lo + up) * step


def _split(x, scale, noise):
    """E2M1 magnitudes (with sign) and exponents of the rows of x, in blocks of 32, zero padded."""
    rows, k = x.shape
    pad = _blocks(k) * 32 - k
    x = torch.nn.functional.pad(x.to(torch.float32), (0, pad)).view(rows, -1, 32)
    noise = None if noise is None else torch.nn.functional.pad(noise, (0, pad)).view(rows, -1, 32)
    e = _exponent(x.abs().amax(-1), scale)
    q = _round(x.abs() / _pow2(e).unsqueeze(-1), noise)
    return torch.copysign(q, x), e


def _values(x, scale, noise):
    q, e = _split(x, scale, noise)
    v = q * _pow2(e).unsqueeze(-1)
    return v.view(x.shape[0], -1)[:, : x.shape[1]]


def _pack(x):
    """An MXFP4 matrix (floor scales, nearest) of the rows of x, laid out as the library takes it."""
    q, e = _split(x, "floor", None)
    rows, nb = e.shape
    mag = q.abs()
    code = torch.where(mag < 2, mag * 2, torch.where(mag < 4, mag + 2, mag / 2 + 4)).to(torch.uint8)
    code = (code + 8 * torch.signbit(q).to(torch.uint8)).view(rows, nb * 16, 2)
    data = code[:, :, 0] + 16 * code[:, :, 1]
    rt, kt = -(-rows // 128), -(-nb // 4)
    s = torch.nn.functional.pad((e + 127).to(torch.uint8), (0, kt * 4 - nb, 0, rt * 128 - rows))
    return data.contiguous(), s.view(rt, 4, 32, kt, 4).permute(0, 3, 2, 1, 4).reshape(-1).contiguous()


def _unpack(q, rows, k):
    data, scales = q
    nb = _blocks(k)
    rt, kt = -(-rows // 128), -(-nb // 4)
    grid = torch.tensor([0, .5, 1, 1.5, 2, 3, 4, 6, -0.0, -.5, -1, -1.5, -2, -3, -4, -6], device=data.device)
    v = grid[torch.stack((data & 15, data >> 4), -1).to(torch.int32)].view(rows, nb, 32)
    e = scales.view(rt, kt, 32, 4, 4).permute(0, 3, 2, 1, 4).reshape(rt * 128, kt * 4)[:rows, :nb].to(torch.int32) - 127
    return (v * _pow2(e).unsqueeze(-1)).view(rows, nb * 32)[:, :k]


def _mx_empty(rows, k):
    tiles = (-(-rows // 128)) * (-(-_blocks(k) // 4))
    return (torch.empty((rows, _blocks(k) * 16), dtype=torch.uint8, device="cuda"),
            torch.empty(tiles * 512, dtype=torch.uint8, device="cuda"))


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
    s = {"case": case}
    if case["op"] == "quantize":
        rows, cols, dt = case["rows"], case["cols"], DTYPES[case["dtype"]]
        s["x"] = _activations((rows, cols), g, dt)
        s["noise"] = torch.randint(0, 256, (rows, cols), generator=g, device="cuda", dtype=torch.uint8) if case["noise"] else None
        r, c = case["dirs"] in ("rows", "both"), case["dirs"] in ("cols", "both")
        s["by_rows"] = _mx_empty(rows, cols) if r else None
        s["by_cols"] = _mx_empty(cols, rows) if c else None
        s["rows_out"] = torch.empty((rows, cols), dtype=dt, device="cuda") if r else None
        s["cols_out"] = torch.empty((cols, rows), dtype=dt, device="cuda") if c else None
        return s
    if case["op"] == "gemm":
        m, n, k = case["m"], case["n"], case["k"]
        s["a"] = _pack(_activations((m, k), g, torch.float32))
        s["b"] = _pack(torch.randn((n, k), generator=g, device="cuda") / math.sqrt(k))
        s["alpha"] = 0.5 if case["beta"] else 1.0
        s["out"] = torch.randn((m, n), generator=g, device="cuda").to(DTYPES[case["out"]])
        return s
    rows, cols, dt = case["rows"], case["cols"], DTYPES[case["dtype"]]
    s["x"] = _activations((rows, cols), g, dt, 0.5)
    s["f"] = _activations((rows, cols), g, dt, 0.5)
    s["post_w"] = 1 + 0.2 * torch.randn(cols, generator=g, device="cuda")
    s["pre_w"] = 1 + 0.2 * torch.randn(cols, generator=g, device="cuda")
    groups = -(-rows // case["per_gate"])
    s["gate"] = torch.randn((groups, cols), generator=g, device="cuda") if case["gate"] else None
    s["res"] = 1 + 0.1 * torch.randn(cols, generator=g, device="cuda") if case["res"] else None
    s["y"], s["h"] = torch.empty_like(s["x"]), torch.empty_like(s["x"])
    s["rstd"] = torch.empty((2, rows), device="cuda")
    if case["op"] == "norm_bwd":
        y, h, rstd = _norm_fwd(s)
        s["y"], s["rstd"], s["h"] = y, rstd, None
        s["dy"] = _activations((rows, cols), g, dt, 0.5)
        s["dh"] = _activations((rows, cols), g, dt, 0.5)
        s["dx"], s["df"] = torch.empty_like(s["x"]), torch.empty_like(s["x"])
        s["d_post_w"], s["d_pre_w"] = torch.empty(cols, device="cuda"), torch.empty(cols, device="cuda")
        s["d_gate"] = torch.empty_like(s["gate"]) if case["gate"] else None
        s["d_res"] = torch.empty(cols, device="cuda") if case["res"] else None
    return s


# ------------------------------------------------------------ plain norms

def _gate_rows(s):
    """The gate of every row."""
    at = torch.arange(s["case"]["rows"], device="cuda") // s["case"]["per_gate"]
    return s["gate"][at]


def _norm_fwd(s):
    x, f = s["x"].to(torch.float32), s["f"].to(torch.float32)
    r1 = torch.rsqrt((f * f).mean(-1, keepdim=True) + EPS)
    n1 = f * r1 * s["post_w"]
    if s["gate"] is not None:
        n1 = n1 * _gate_rows(s)
    y = n1 + (x if s["res"] is None else x * s["res"])
    r2 = torch.rsqrt((y * y).mean(-1, keepdim=True) + EPS)
    return y.to(s["x"].dtype), (y * r2 * s["pre_w"]).to(s["x"].dtype), torch.stack((r1[:, 0], r2[:, 0]))


def _norm_bwd(s):
    x, f, y = s["x"].to(torch.float32), s["f"].to(torch.float32), s["y"].to(torch.float32)
    dy, dh = s["dy"].to(torch.float32), s["dh"].to(torch.float32)
    r1, r2 = s["rstd"][0].unsqueeze(1), s["rstd"][1].unsqueeze(1)
    yn, fn = y * r2, f * r1
    g2 = dh * s["pre_w"]
    dyt = dy + r2 * (g2 - yn * (g2 * yn).mean(-1, keepdim=True))
    dx = dyt if s["res"] is None else dyt * s["res"]
    dn = dyt if s["gate"] is None else dyt * _gate_rows(s)
    g1 = dn * s["post_w"]
    df = r1 * (g1 - fn * (g1 * fn).mean(-1, keepdim=True))
    d_gate = None
    if s["gate"] is not None:
        at = torch.arange(x.shape[0], device="cuda") // s["case"]["per_gate"]
        d_gate = torch.zeros_like(s["gate"]).index_add_(0, at, dyt * fn * s["post_w"])
    return {"dx": dx.to(s["x"].dtype), "df": df.to(s["x"].dtype), "d_post_w": (dn * fn).sum(0), "d_pre_w": (dh * yn).sum(0),
            "d_gate": d_gate, "d_res": None if s["res"] is None else (dyt * x).sum(0)}


# ------------------------------------------------------------ run

_kept = {}


def _handle():
    if "h" not in _kept:
        import newton_schulz_nesterov_gb300 as dm
        _kept["dm"], _kept["h"] = dm, dm.Handle(0)
    return _kept["h"]


def _run_own(s):
    h, case = _handle(), s["case"]
    if case["op"] == "quantize":
        h.mxfp4_quantize(s["x"], by_rows=s["by_rows"], by_cols=s["by_cols"], noise=s["noise"], scale=case["scale"])
        if s["by_rows"] is not None:
            h.mxfp4_dequantize(s["by_rows"], s["rows_out"])
        if s["by_cols"] is not None:
            h.mxfp4_dequantize(s["by_cols"], s["cols_out"])
        return {"rows": s["rows_out"], "cols": s["cols_out"]}
    if case["op"] == "gemm":
        h.mxfp4_gemm(s["a"], s["b"], s["out"], case["k"], alpha=s["alpha"], beta=case["beta"])
        return s["out"]
    if case["op"] == "norm_fwd":
        h.block_norm_forward(s["x"], s["f"], s["post_w"], s["pre_w"], s["y"], s["h"], s["rstd"], gate=s["gate"],
                             rows_per_gate=case["per_gate"], res_scale=s["res"], eps=EPS)
        return {"y": s["y"], "h": s["h"], "rstd": s["rstd"]}
    h.block_norm_backward(s["dy"], s["dh"], s["x"], s["f"], s["y"], s["post_w"], s["pre_w"], s["rstd"], s["dx"], s["df"],
                          s["d_post_w"], s["d_pre_w"], gate=s["gate"], d_gate=s["d_gate"], rows_per_gate=case["per_gate"],
                          res_scale=s["res"], d_res_scale=s["d_res"])
    return {k: s[k] for k in ("dx", "df", "d_post_w", "d_pre_w", "d_gate", "d_res")}


def run(s):
    if own:
        return _run_own(s)
    case = s["case"]
    if case["op"] == "quantize":
        x, noise = s["x"], s["noise"]
        return {"rows": None if s["by_rows"] is None else _values(x, case["scale"], noise).to(x.dtype),
                "cols": None if s["by_cols"] is None else
                _values(x.t(), case["scale"], None if noise is None else noise.t()).to(x.dtype)}
    if case["op"] == "gemm":
        d = s["alpha"] * (_unpack(s["a"], case["m"], case["k"]) @ _unpack(s["b"], case["n"], case["k"]).t())
        if case["beta"]:
            d = d + case["beta"] * s["out"].to(torch.float32)
        s["out"].copy_(d)
        return s["out"]
    if case["op"] == "norm_fwd":
        y, h, rstd = _norm_fwd(s)
        return {"y": y, "h": h, "rstd": rstd}
    return _norm_bwd(s)


# ------------------------------------------------------------ 64 bits

def exact(case, seed):
    s = prepare(case, seed)
    dev, f64 = "cuda", torch.float64

    def two_to(e):
        return ((e.to(torch.int64) + 1023) << 52).view(f64)

    def read_back(x, noise):
        """Rows of x quantised and read back, by comparing with every value of the grid."""
        rows, k = x.shape
        wide = -(-k // 32) * 32
        grid = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)
        out = torch.empty((rows, k), dtype=f64, device=dev)
        per = max(1, (1 << 25) // wide)
        for i in range(0, rows, per):
            part = x[i:i + per].to(f64)
            full = torch.zeros((part.shape[0], wide), dtype=f64, device=dev)
            full[:, :k] = part
            b = full.view(part.shape[0], -1, 32)
            top = b.abs().amax(-1, keepdim=True)
            safe = torch.where(top > 0, top, torch.ones_like(top))
            if case["scale"] == "floor":  # 4 * 2^e <= top < 8 * 2^e
                e = torch.floor(torch.log2(safe)) - 2
                e = e + (safe >= 8 * two_to(e)).to(f64) - (safe < 4 * two_to(e)).to(f64)
            else:  # 3 * 2^e < top <= 6 * 2^e
                e = torch.ceil(torch.log2(safe / 6))
                e = e + (safe > 6 * two_to(e)).to(f64) - (safe <= 3 * two_to(e)).to(f64)
            unit = two_to(torch.where(top > 0, e, torch.full_like(e, -127)).clamp(-127, 127))
            v = (b.abs() / unit).clamp(max=6.0)
            if noise is not None:
                z = torch.zeros_like(full)
                z[:, :k] = noise[i:i + per].to(f64)
                z = z.view_as(v)
            q = torch.zeros_like(v)
            for j in range(7):
                lo, hi = grid[j], grid[j + 1]
                if noise is not None:
                    up = (v - lo) / (hi - lo) > (z + 0.5) / 256
                else:
                    up = (v >= (lo + hi) / 2) if j % 2 else (v > (lo + hi) / 2)
                q = torch.where(v >= lo, torch.where(up, hi, lo).to(f64), q)
            q = torch.where(v >= 6.0, torch.full_like(q, 6.0), q)
            out[i:i + per] = (torch.copysign(q, b) * unit).view(part.shape[0], -1)[:, :k]
        return out

    def decoded(q, rows, k):
        """An MXFP4 matrix in 64 bits, from the bits of its codes."""
        code = torch.empty((rows, q[0].shape[1] * 2), dtype=torch.int32, device=dev)
        code[:, 0::2], code[:, 1::2] = q[0] % 16, q[0] // 16
        exp, man = (code // 2) % 4, (code % 2).to(f64)
        mag = torch.where(exp == 0, man / 2, (1 + man / 2) * two_to(exp - 1))
        r, j = torch.arange(rows, device=dev)[:, None], torch.arange(q[0].shape[1] // 16, device=dev)[None, :]
        at = ((r // 128) * (-(-q[0].shape[1] // 64)) + j // 4) * 512 + (r % 32) * 16 + (r % 128) // 32 * 4 + j % 4
        unit = two_to(q[1][at].to(torch.int64) - 127)
        return (torch.where(code >= 8, -mag, mag).view(rows, -1, 32) * unit[:, :, None]).view(rows, -1)[:, :k]

    if case["op"] == "quantize":
        return {"rows": read_back(s["x"], s["noise"]) if s["by_rows"] is not None else None,
                "cols": read_back(s["x"].t(), None if s["noise"] is None else s["noise"].t())
                if s["by_cols"] is not None else None}
    if case["op"] == "gemm":
        d = decoded(s["a"], case["m"], case["k"]) @ decoded(s["b"], case["n"], case["k"]).t()
        return d.mul_(s["alpha"]).add_(s["out"].to(f64), alpha=case["beta"])
    t = {k: (v.to(f64) if isinstance(v, torch.Tensor) else v) for k, v in s.items()}
    cols, per = case["cols"], case["per_gate"]
    gate = t["gate"].repeat_interleave(per, 0)[: case["rows"]] if t["gate"] is not None else 1.0
    res = 1.0 if t["res"] is None else t["res"]
    if case["op"] == "norm_fwd":
        r1 = (t["f"].square().sum(-1) / cols + EPS) ** -0.5
        y = res * t["x"] + gate * (t["post_w"] * (t["f"] * r1[:, None]))
        r2 = (y.square().sum(-1) / cols + EPS) ** -0.5
        return {"y": y, "h": t["pre_w"] * (y * r2[:, None]), "rstd": torch.stack((r1, r2))}
    r1, r2 = t["rstd"][0][:, None], t["rstd"][1][:, None]
    into = t["dh"] * t["pre_w"] * r2
    dyt = t["dy"] + into - t["y"] * (into * t["y"]).sum(-1, keepdim=True) * r2 ** 2 / cols
    back = gate * dyt * t["post_w"] * r1
    df = back - t["f"] * (back * t["f"]).sum(-1, keepdim=True) * r1 ** 2 / cols
    each = dyt * t["f"] * r1
    d_gate = None
    if t["gate"] is not None:
        pad = t["gate"].shape[0] * per - case["rows"]
        d_gate = torch.nn.functional.pad(each * t["post_w"], (0, 0, 0, pad)).view(-1, per, cols).sum(1)
    return {"dx": res * dyt, "df": df, "d_post_w": (gate * each).sum(0), "d_pre_w": (t["dh"] * t["y"] * r2).sum(0),
            "d_gate": d_gate, "d_res": None if t["res"] is None else (dyt * t["x"]).sum(0)}
