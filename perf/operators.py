"""The 8-bit (MX) operators of the denoiser's blocks: what is measured of them.

Values in MX form are e4m3 with one power-of-two scale (e8m0) for each 32
consecutive values of a row: e is the smallest integer with
max |x| <= 448 * 2^e (at least -127), and the stored value is x * 2^-e rounded
to e4m3.  The scales lie in tiles of 128 rows x 4 blocks:
scale[r // 128, b // 4, r % 32, r % 128 // 32, b % 4] for row r and block b.
"""

import math

import torch

own = False

HEADS = 32
WIDTH = 128 * HEADS      # hidden width of the denoiser's blocks
HIDDEN = 3 * WIDTH       # the SwiGLU layer is three times as wide
EPS = 1e-6


def listed():
    return [
        # a short prompt's attention output, in front of the output projection: latency
        dict(name="quantize prompt", op="quantize", M=16, K=WIDTH),
        # the attention output of the text-to-image layout's first step (256 text + 64x64 target tokens)
        dict(name="quantize t2i", op="quantize", M=4352, K=WIDTH),
        # the norm in front of a projection, an odd number of prompt tokens, with the residual's addition: latency
        dict(name="norm prompt", op="norm", M=37, K=WIDTH, residual=True),
        # the same over every token of the layout with ten reference images
        dict(name="norm maxref", op="norm", M=28160, K=WIDTH, residual=True),
        # first layer of a time-embedding MLP: one row, 256 sinusoids, SiLU: the smallest call
        dict(name="linear time", op="linear", M=1, N=WIDTH, K=256, n_out=1, act="silu", bias=True, residual=False),
        # one row against a large weight: six modulation vectors of a block from the step's embedding
        dict(name="linear modulation", op="linear", M=1, N=6 * WIDTH, K=WIDTH, n_out=1, act="none", bias=True,
             residual=False),
        # an odd number of prompt tokens through a text projection with GELU
        dict(name="linear text", op="linear", M=333, N=WIDTH, K=WIDTH, n_out=1, act="gelu", bias=True, residual=False),
        # fused Q/K/V projection of a 64x64 target
        dict(name="linear qkv", op="linear", M=4096, N=3 * WIDTH, K=WIDTH, n_out=3, act="none", bias=True,
             residual=False),
        # the feed-forward layer's down projection with the residual, text-to-image layout, first step
        dict(name="linear down", op="linear", M=4352, N=WIDTH, K=HIDDEN, n_out=1, act="none", bias=True, residual=True),
        # the gated half of the feed-forward layer: a short odd prompt, a 64x64 target, a 128x128 target
        dict(name="swiglu prompt", op="swiglu", M=77, N=HIDDEN, K=WIDTH),
        dict(name="swiglu t2i", op="swiglu", M=4096, N=HIDDEN, K=WIDTH),
        dict(name="swiglu hires", op="swiglu", M=16384, N=HIDDEN, K=WIDTH),
    ]


def draw(rng):
    def spread(lo, hi):
        return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))

    op = rng.choice(("quantize", "norm", "linear", "linear", "swiglu"))
    M, K = spread(1, 28160), 32 * spread(2, 384)
    if op == "quantize":
        return dict(op=op, M=M, K=K)
    if op == "norm":
        return dict(op=op, M=M, K=K, residual=rng.random() < 0.5)
    if op == "linear":
        n_out = rng.choice((1, 1, 3))
        N = n_out * 8 * spread(4, 1536 if n_out == 1 else 512)
        case = dict(op=op, M=M, N=N, K=K, n_out=n_out, act=rng.choice(("none", "silu", "gelu")),
                    bias=rng.random() < 0.7, residual=n_out == 1 and rng.random() < 0.5)
        per_row = 2 * N * K
    else:
        case = dict(op=op, M=M, N=128 * spread(1, 96), K=K)
        per_row = 4 * case["N"] * K
    most = 4 * 16384 * HIDDEN * WIDTH
    case["M"] = max(1, min(M, most // per_row))
    return case


# ------------------------------------------------------------- the plain form

def _tile(s):
    """Scale bytes [R, B] -> [ceil(R / 128), ceil(B / 4), 32, 4, 4], zero padded."""
    R, B = s.shape
    rt, bt = -(-R // 128), -(-B // 4)
    t = torch.zeros(rt * 128, bt * 4, dtype=torch.uint8, device=s.device)
    t[:R, :B] = s
    return t.view(rt, 4, 32, bt, 4).permute(0, 3, 2, 1, 4).contiguous()


def _untile(t, R, B):
    rt, bt = t.shape[:2]
    return t.view(torch.uint8).permute(0, 3, 2, 1, 4).reshape(rt * 128, bt * 4)[:R, :B]


def _quantize(x):
    """float32 [R, K] -> (e4m3 [R, K], tiled e8m0)."""
    R, K = x.shape
    blocks = x.view(R, K // 32, 32)
    m, e = torch.frexp(blocks.abs().amax(-1))  # amax = m * 2^e, 1/2 <= m < 1; 448 = 7/8 * 2^9
    e = torch.where(m > 0.875, e - 8, e - 9).clamp_min(-127)
    e = torch.where(m == 0, torch.full_like(e, -127), e)
    q = torch.ldexp(blocks, -e[..., None]).view(R, K).to(torch.float8_e4m3fn)
    return q, _tile((e + 127).to(torch.uint8)).view(torch.float8_e8m0fnu)


def _values(q, scale):
    R, K = q.shape
    s = torch.exp2(_untile(scale, R, K // 32).float() - 127)
    return (q.float().view(R, K // 32, 32) * s[..., None]).view(R, K)


def _product(x, w, bias):
    y = _values(*x) @ _values(*w).t()
    return y if bias is None else y + bias.float()


def _plain(s):
    c, op = s["case"], s["case"]["op"]
    if op == "quantize":
        q, scale = _quantize(s["x"].float())
        return dict(q=q, scale=scale)
    if op == "norm":
        h = s["x"]
        got = {}
        if c["residual"]:
            h = got["sum"] = (h.float() + s["delta"].float()).to(torch.bfloat16)
        h = h.float()
        y = h * torch.rsqrt(h.square().mean(-1, keepdim=True) + EPS) * s["w"].float()
        got["q"], got["scale"] = _quantize(y)
        return got
    if op == "linear":
        y = _product(s["x"], s["w"], s["bias"])
        if c["act"] == "silu":
            y = y / (1 + torch.exp(-y))
        elif c["act"] == "gelu":
            y = 0.5 * y * (1 + torch.tanh(math.sqrt(2 / math.pi) * (y + 0.044715 * y * y * y)))
        if c["residual"]:
            y = s["residual"].float() + s["alpha"] * y
        return [t.contiguous() for t in y.to(torch.bfloat16).chunk(c["n_out"], dim=1)]
    y = _product(s["x"], s["w"], s["bias"]).view(c["M"], c["N"] // 128, 2, 128)
    g, u = y[:, :, 0], y[:, :, 1]
    q, scale = _quantize((g / (1 + torch.exp(-g)) * u).reshape(c["M"], c["N"]))
    return dict(q=q, scale=scale)


# -------------------------------------------------------------- the framework

def _framework(s):
    import diffusion_transformer_joint_axial_b200 as qi

    c, op = s["case"], s["case"]["op"]
    if op == "quantize":
        t = qi.mx_quantize(s["x"], out=qi.MXTensor(*s["out"]))
        return dict(q=t.q, scale=t.scale)
    if op == "norm":
        if c["residual"]:
            h, t = qi.rmsnorm_mx(s["x"], s["w"], EPS, delta=s["delta"], sum_out=s["sum"], out=qi.MXTensor(*s["out"]))
            return dict(sum=h, q=t.q, scale=t.scale)
        t = qi.rmsnorm_mx(s["x"], s["w"], EPS, out=qi.MXTensor(*s["out"]))
        return dict(q=t.q, scale=t.scale)
    x, w = qi.MXTensor(*s["x"]), qi.MXTensor(*s["w"])
    if op == "linear":
        return qi.linear_mx(x, w, s["bias"], n_out=c["n_out"], act=c["act"], residual=s["residual"], alpha=s["alpha"],
                            out=s["out"], workspace=s["workspace"])
    t = qi.linear_swiglu_mx(x, w, s["bias"], out=qi.MXTensor(*s["out"]), workspace=s["workspace"])
    return dict(q=t.q, scale=t.scale)


def run(state):
    return _framework(state) if own else _plain(state)


# ------------------------------------------------------------------ the inputs

def _activations(gen, M, K):
    """Rows of normal values whose channels differ in size, as a residual stream's do."""
    channel = torch.exp(0.5 * torch.randn(K, generator=gen, device="cuda"))
    return torch.randn(M, K, generator=gen, device="cuda").mul_(channel).to(torch.bfloat16)


def _empty_mx(M, K):
    return (torch.empty(M, K, dtype=torch.float8_e4m3fn, device="cuda"),
            torch.zeros(-(-M // 128), -(-K // 128), 32, 4, 4, dtype=torch.uint8,
                        device="cuda").view(torch.float8_e8m0fnu))


def prepare(case, seed):
    c = case
    gen = torch.Generator(device="cuda").manual_seed(int(seed))
    M, K = c["M"], c["K"]
    s = dict(case=c)
    if c["op"] == "quantize":
        return dict(s, x=_activations(gen, M, K), out=_empty_mx(M, K))
    if c["op"] == "norm":
        s.update(x=_activations(gen, M, K), out=_empty_mx(M, K),
                 w=(1 + 0.1 * torch.randn(K, generator=gen, device="cuda")).to(torch.bfloat16))
        if c["residual"]:
            s.update(delta=(0.3 * torch.randn(M, K, generator=gen, device="cuda")).to(torch.bfloat16),
                     sum=torch.empty(M, K, dtype=torch.bfloat16, device="cuda"))
        return s
    N = c["N"] * (2 if c["op"] == "swiglu" else 1)
    s["x"] = _quantize(_activations(gen, M, K).float())
    s["w"] = _quantize(torch.randn(N, K, generator=gen, device="cuda") / math.sqrt(K))
    bias = (0.1 * torch.randn(N, generator=gen, device="cuda")).to(torch.bfloat16)
    s["workspace"] = torch.zeros(256, dtype=torch.uint8, device="cuda")
    if c["op"] == "swiglu":
        return dict(s, bias=bias, out=_empty_mx(M, c["N"]))
    s.update(bias=bias if c["bias"] else None, residual=None, alpha=1.0)
    if c["residual"]:
        s.update(residual=torch.randn(M, N, generator=gen, device="cuda").to(torch.bfloat16), alpha=0.75)
    s["out"] = [torch.empty(M, N // c["n_out"], dtype=torch.bfloat16, device="cuda") for _ in range(c["n_out"])]
    return s


def work(case):
    c = case
    M, K = c["M"], c["K"]
    if c["op"] == "quantize":
        return {"bytes": M * K * (2 + 33 / 32), "flops": 2 * M * K}
    if c["op"] == "norm":
        return {"bytes": M * K * (2 + 33 / 32 + (4 if c["residual"] else 0)) + 2 * K, "flops": 5 * M * K}
    if c["op"] == "linear":
        N = c["N"]
        return {"bytes": (M + N) * K * 33 / 32 + M * N * (4 if c["residual"] else 2) + (2 * N if c["bias"] else 0),
                "flops": 2 * M * N * K}
    N = 2 * c["N"]
    return {"bytes": (M + N) * K * 33 / 32 + M * c["N"] * 33 / 32 + 2 * N, "flops": 2 * M * N * K}


# ----------------------------------------------- the definition, in 64 bits

def _wide(mx):
    """The float64 values that an MX tensor stands for, element by element."""
    q, scale = mx
    R, K = q.shape
    r = torch.arange(R, device=q.device)[:, None]
    b = torch.arange(K // 32, device=q.device)[None, :]
    byte = scale.view(torch.uint8)[r // 128, b // 4, r % 32, r % 128 // 32, b % 4]
    step = torch.pow(torch.tensor(2.0, dtype=torch.float64, device=q.device), byte.double() - 127.0)
    return q.double() * step.repeat_interleave(32, dim=1)


def _stored(y):
    """The values in front of their rounding to 8 bits: y over its block's power of two.  The power itself is a
    choice of the storage, not a computed number."""
    R, K = y.shape
    top = y.reshape(R, K // 32, 32).abs().max(-1).values
    ratio = torch.clamp(top / 448.0, min=2.0 ** -127)
    e = torch.round(torch.log2(ratio))
    power = torch.where(torch.pow(2.0, e) >= ratio, torch.pow(2.0, e), torch.pow(2.0, e + 1))
    power = torch.where(torch.pow(2.0, e - 1) >= ratio, torch.pow(2.0, e - 1), power)
    return dict(q=y / power.repeat_interleave(32, dim=1), scale=None)


def exact(case, seed):
    c = case
    s = prepare(case, seed)
    if c["op"] == "quantize":
        return _stored(s["x"].double())
    if c["op"] == "norm":
        got = {}
        h = s["x"].double()
        if c["residual"]:
            got["sum"] = h + s["delta"].double()
            h = got["sum"].to(torch.bfloat16).double()  # the norm is that of the stored sum
        ms = torch.sum(h * h, dim=1, keepdim=True) / c["K"]
        got.update(_stored(h / torch.sqrt(ms + EPS) * s["w"].double()))
        return got
    y = torch.mm(_wide(s["x"]), _wide(s["w"]).T)
    if s["bias"] is not None:
        y += s["bias"].double()
    if c["op"] == "linear":
        if c["act"] == "silu":
            y *= torch.sigmoid(y)
        elif c["act"] == "gelu":
            y *= torch.sigmoid(2.0 * math.sqrt(2.0 / math.pi) * (y + 0.044715 * y ** 3))
        if c["residual"]:
            y = s["residual"].double() + s["alpha"] * y
        w = c["N"] // c["n_out"]
        return [y[:, i * w:(i + 1) * w] for i in range(c["n_out"])]
    M, F = c["M"], c["N"]
    m = torch.empty(M, F, dtype=torch.float64, device=y.device)
    for j in range(F // 128):
        g, u = y[:, 256 * j:256 * j + 128], y[:, 256 * j + 128:256 * j + 256]
        m[:, 128 * j:128 * j + 128] = g * torch.sigmoid(g) * u
    return _stored(m)
