"""The operators around a quantized linear layer, as measured cases: the
block-scaled GEMM with an epilogue (bias, activation, dropout, residual), the
backward of that epilogue, layer norm forward and backward, and dropout.

``run`` computes a case in plain torch operations (``own`` false) or by the
library's calls (``own`` true); ``exact`` gives the same results in 64 bits.
"""
import math

import torch

own = False

DEV = "cuda"
DTYPES = {"bf16": torch.bfloat16, "f32": torch.float32}
FMTS = {"mxfp4": 0, "nvfp4": 1, "mxfp8": 2}
ACTS = {"none": 0, "relu": 1, "gelu": 2, "gelu_tanh": 3, "silu": 4}
GROUP = {"mxfp4": 32, "nvfp4": 16, "mxfp8": 32}
E2M1 = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)


# ------------------------------------------------------------------ cases
def _gemm(fmt, M, N, K, out="bf16", bias="bf16", act="none", preact=False, p=0.0, residual=None):
    return {"op": "gemm_epilogue", "fmt": fmt, "M": M, "N": N, "K": K, "out": out, "bias": bias, "act": act,
            "preact": preact, "p": p, "residual": residual}


def listed():
    return [
        # one token through a projection that is kept in MXFP8 (serving, latency)
        dict(_gemm("mxfp8", 1, 4096, 4096), name="gemm_token_mxfp8"),
        # a batch of decoding sequences through an up projection (serving)
        dict(_gemm("mxfp4", 100, 11008, 4096, act="silu"), name="gemm_decode_mxfp4"),
        # a training step's up projection: bias and GELU, the sum before the GELU kept for the backward pass
        dict(_gemm("nvfp4", 8192, 11008, 4096, act="gelu", preact=True), name="gemm_up_nvfp4"),
        # a training step's down projection: bias, dropout, added to the residual stream
        dict(_gemm("nvfp4", 16384, 4096, 14336, p=0.1, residual="bf16"), name="gemm_down_nvfp4"),
        # the way back through the up projection's GELU and bias
        {"name": "epilogue_backward_up", "op": "epilogue_backward", "M": 8192, "N": 11008, "dt": "bf16", "act": "gelu",
         "p": 0.0},
        # a short last batch in binary32, with dropout
        {"name": "epilogue_backward_ragged", "op": "epilogue_backward", "M": 515, "N": 1001, "dt": "f32",
         "act": "silu", "p": 0.2},
        # the norm before a layer: a few tokens of a serving step, and a training step's activations
        {"name": "layernorm_tokens", "op": "layernorm_forward", "M": 4, "D": 4096, "dt": "bf16", "wdt": "bf16"},
        {"name": "layernorm_train", "op": "layernorm_forward", "M": 16384, "D": 4096, "dt": "bf16", "wdt": "f32"},
        # its backward pass with the gradients of weight and bias; an odd width in binary32
        {"name": "layernorm_backward_train", "op": "layernorm_backward", "M": 8192, "D": 4096, "dt": "bf16",
         "wdt": "f32"},
        {"name": "layernorm_backward_odd", "op": "layernorm_backward", "M": 509, "D": 1001, "dt": "f32", "wdt": "f32"},
        # dropout of a block's output onto the residual stream; dropout alone (or its backward) on an odd count
        {"name": "dropout_residual", "op": "dropout", "n": 16384 * 4096, "dt": "bf16", "p": 0.1, "residual": True},
        {"name": "dropout_odd", "op": "dropout", "n": 515 * 1001, "dt": "f32", "p": 0.5, "residual": False},
    ]


def _log(rng, lo, hi, step=1):
    return max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi))) / step)) * step)


def draw(rng):
    op = rng.choice(["gemm_epilogue", "gemm_epilogue", "epilogue_backward", "layernorm_forward", "layernorm_backward",
                     "dropout"])
    dt = rng.choice(["bf16", "bf16", "f32"])
    p = rng.choice([0.0, rng.uniform(0.02, 0.6)])
    if op == "gemm_epilogue":
        while True:
            M, N, K = _log(rng, 1, 16384), _log(rng, 8, 14336, 8), _log(rng, 32, 14336, 32)
            if 1 << 20 <= M * N * K <= 8192 * 11008 * 4096:
                break
        fmt = rng.choice(list(FMTS))
        # sums of FP4 products are exact to binary32; the tensor cores' E4M3 sums are not, so MXFP8 goes to bf16
        return _gemm(fmt, M, N, K, out="bf16" if fmt == "mxfp8" else dt, bias=rng.choice([None, "bf16", "f32"]),
                     act=rng.choice(list(ACTS)), preact=rng.choice([False, True]), p=p,
                     residual=rng.choice([None, "bf16", "f32"]))
    if op == "dropout":
        return {"op": op, "n": _log(rng, 4096, 1 << 26), "dt": dt, "p": p or 0.1, "residual": rng.choice([False, True])}
    while True:
        M, W = _log(rng, 1, 16384), _log(rng, 16, 16384)
        W = W if rng.random() < 0.4 else (W + 15) // 16 * 16
        if 4096 <= M * W <= 1 << 26:
            break
    if op == "epilogue_backward":
        return {"op": op, "M": M, "N": W, "dt": dt, "act": rng.choice(list(ACTS)), "p": p}
    return {"op": op, "M": M, "D": W, "dt": dt, "wdt": rng.choice(["bf16", "f32"])}


def work(case):
    op = case["op"]
    size = {"bf16": 2, "f32": 4, None: 0}
    if op == "gemm_epilogue":
        M, N, K, fmt = case["M"], case["N"], case["K"], case["fmt"]
        codes = 1.0 if fmt == "mxfp8" else 0.5
        b = (M + N) * K * (codes + 1.0 / GROUP[fmt]) + N * size[case["bias"]]
        b += M * N * (size[case["out"]] * (2 if case["preact"] else 1) + size[case["residual"]])
        return {"bytes": b, "flops": 2.0 * M * N * K}
    if op == "dropout":
        return {"bytes": case["n"] * size[case["dt"]] * (3 if case["residual"] else 2), "flops": 2.0 * case["n"]}
    s = size[case["dt"]]
    if op == "epilogue_backward":
        n = case["M"] * case["N"]
        return {"bytes": n * s * (2 if case["act"] == "none" else 3) + 4 * case["N"], "flops": 4.0 * n}
    n, w = case["M"] * case["D"], case["D"] * size[case["wdt"]]
    if op == "layernorm_forward":
        return {"bytes": 2 * n * s + 2 * w + 8 * case["M"], "flops": 8.0 * n}
    return {"bytes": 3 * n * s + w + 8 * case["M"] + 8 * case["D"], "flops": 14.0 * n}


# ------------------------------------------------------------------ inputs
def _blocks(x, fmt):
    """Codes, scales and tensor scale of x (rows, K), in the layouts the library's quantize calls write."""
    rows, K = x.shape
    g = GROUP[fmt]
    xb = x.view(rows, K // g, g)
    amax = xb.abs().amax(-1)
    ts = None
    if fmt == "nvfp4":
        ts = (amax.max() / 2688.0).reshape(1)
        s8 = (amax / 6.0 / ts).to(torch.float8_e4m3fn)
        scales, S = s8.view(torch.uint8), s8.float() * ts
    else:
        k = torch.ceil(torch.log2(amax / (448.0 if fmt == "mxfp8" else 6.0))).clamp(-126, 127)
        scales, S = (k + 127).to(torch.uint8), torch.exp2(k)
    v = xb / S.clamp_min(1e-38)[..., None]
    if fmt == "mxfp8":
        codes = v.clamp(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8).reshape(rows, K)
    else:
        mid = torch.tensor([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0], device=x.device)
        c = torch.bucketize(v.abs(), mid).to(torch.uint8) + (v < 0).to(torch.uint8) * 8
        c = c.view(rows, K // 2, 2)
        codes = c[..., 0] | (c[..., 1] << 4)
    out = {"codes": codes.contiguous(), "scales": scales.contiguous()}
    if ts is not None:
        out["tscale"] = ts
    return out


def prepare(case, seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)

    def normal(shape, std=1.0, dt="f32"):
        return (torch.randn(shape, generator=g, device=DEV) * std).to(DTYPES[dt])

    op, s = case["op"], dict(case)
    s["seed"] = 1_000_003 * seed + 17
    s["step"] = torch.tensor([seed % 1000], dtype=torch.int64, device=DEV)   # a training loop's step counter
    if op == "gemm_epilogue":
        M, N, K = case["M"], case["N"], case["K"]
        x = normal((M, K))
        x[:, torch.randperm(K, generator=g, device=DEV)[:max(1, K // 100)]] *= 20.0   # outlier channels
        s["A"] = _blocks(x, case["fmt"])
        s["B"] = _blocks(normal((N, K), 0.02 * math.sqrt(4096 / K)), case["fmt"])
        s["bias_t"] = normal((N,), 0.5, case["bias"]) if case["bias"] else None
        s["residual_t"] = normal((M, N), 2.0, case["residual"]) if case["residual"] else None
    elif op == "epilogue_backward":
        s["dy"] = normal((case["M"], case["N"]), 1e-3, case["dt"])
        s["z"] = normal((case["M"], case["N"]), 1.5, case["dt"])
    elif op == "dropout":
        s["x"] = normal((case["n"],), 1.0, case["dt"])
        s["residual_t"] = normal((case["n"],), 2.0, case["dt"]) if case["residual"] else None
    else:
        M, D = case["M"], case["D"]
        s["x"] = (normal((M, D), 1.5) + 0.5 * normal((M, 1)) + 0.3).to(DTYPES[case["dt"]])
        s["gamma"] = (1.0 + normal((D,), 0.2)).to(DTYPES[case["wdt"]])
        s["beta"] = normal((D,), 0.2, case["wdt"])
        if op == "layernorm_backward":
            x = s["x"].double()
            s["mean"] = x.mean(-1).float()
            s["rstd"] = (x.var(-1, unbiased=False) + 1e-5).rsqrt().float()
            s["dy"] = normal((M, D), 1e-3, case["dt"])
    return s


# ------------------------------------------------------------------ plain forms
def _words(n, seed, step):
    """The 32-bit words of elements 0 .. n-1: word e mod 4 of Philox4x32-10, key `seed`, counter (e / 4, 2^63 + step)."""
    lo = 0xFFFFFFFF
    q = torch.arange((n + 3) // 4, device=step.device)
    c0, c1 = q & lo, q >> 32
    c2, c3 = (step & lo).expand_as(q), ((step >> 32) | 0x80000000).expand_as(q)
    k0, k1 = seed & lo, (seed >> 32) & lo
    for _ in range(10):
        p0, p1 = c0 * 0xD2511F53, c2 * 0xCD9E8D57
        c0, c1, c2, c3 = ((p1 >> 32) & lo) ^ c1 ^ k0, p1 & lo, ((p0 >> 32) & lo) ^ c3 ^ k1, p0 & lo
        k0, k1 = (k0 + 0x9E3779B9) & lo, (k1 + 0xBB67AE85) & lo
    return torch.stack([c0, c1, c2, c3], -1).reshape(-1)[:n]


def _drop(v, p, seed, step):
    if p == 0.0:
        return v
    keep = (_words(v.numel(), seed, step) >= int(p * 2.0 ** 32)).view(v.shape)
    return torch.where(keep, v * (1.0 / (1.0 - p)), torch.zeros_like(v))


def _act(z, act):
    if act == "relu":
        return torch.where(z < 0, torch.zeros_like(z), z)
    if act == "gelu":
        return 0.5 * z * (1.0 + torch.erf(z * math.sqrt(0.5)))
    if act == "gelu_tanh":
        return 0.5 * z * (1.0 + torch.tanh(math.sqrt(2.0 / math.pi) * (z + 0.044715 * z * z * z)))
    if act == "silu":
        return z / (1.0 + torch.exp(-z))
    return z


def _act_grad(z, act):
    if act == "relu":
        return (z > 0).to(z.dtype)
    if act == "gelu":
        return 0.5 * (1.0 + torch.erf(z * math.sqrt(0.5))) + z * torch.exp(-0.5 * z * z) / math.sqrt(2.0 * math.pi)
    if act == "gelu_tanh":
        c = math.sqrt(2.0 / math.pi)
        t = torch.tanh(c * (z + 0.044715 * z * z * z))
        return 0.5 * (1.0 + t) + 0.5 * z * (1.0 - t * t) * c * (1.0 + 3 * 0.044715 * z * z)
    if act == "silu":
        s = 1.0 / (1.0 + torch.exp(-z))
        return s * (1.0 + z * (1.0 - s))
    return torch.ones_like(z)


def _values(t, fmt):
    """The numbers that codes and block scales stand for, without the tensor scale, in binary32."""
    rows = t["codes"].shape[0]
    if fmt == "mxfp8":
        v = t["codes"].view(torch.float8_e4m3fn).float()
    else:
        table = torch.tensor(E2M1 + tuple(-v for v in E2M1), device=t["codes"].device)
        v = table[torch.stack([t["codes"] & 15, t["codes"] >> 4], -1).int()]
    if fmt == "nvfp4":
        s = t["scales"].view(torch.float8_e4m3fn).float()
    else:
        s = torch.tensor([2.0 ** (i - 127) for i in range(255)] + [math.nan], device=t["codes"].device)[t["scales"].int()]
    return (v.view(rows, -1, GROUP[fmt]) * s[..., None]).view(rows, -1)


def _plain(s):
    op = s["op"]
    if op == "gemm_epilogue":
        z = _values(s["A"], s["fmt"]) @ _values(s["B"], s["fmt"]).T
        if s["fmt"] == "nvfp4":
            z = z * (s["A"]["tscale"] * s["B"]["tscale"])
        if s["bias_t"] is not None:
            z = z + s["bias_t"].float()
        y = _drop(_act(z, s["act"]), s["p"], s["seed"], s["step"])
        if s["residual_t"] is not None:
            y = y + s["residual_t"].float()
        out = DTYPES[s["out"]]
        return {"y": y.to(out), "preact": z.to(out) if s["preact"] else None}
    if op == "epilogue_backward":
        d = _drop(s["dy"].float(), s["p"], s["seed"], s["step"]) * _act_grad(s["z"].float(), s["act"])
        return {"dz": d.to(s["dy"].dtype), "dbias": d.sum(0)}
    if op == "dropout":
        y = _drop(s["x"].float(), s["p"], s["seed"], s["step"])
        if s["residual_t"] is not None:
            y = y + s["residual_t"].float()
        return {"y": y.to(s["x"].dtype)}
    x = s["x"].float()
    if op == "layernorm_forward":
        mean = x.mean(-1, keepdim=True)
        xc = x - mean
        rstd = 1.0 / torch.sqrt((xc * xc).mean(-1, keepdim=True) + 1e-5)
        y = xc * rstd * s["gamma"].float() + s["beta"].float()
        return {"y": y.to(s["x"].dtype), "mean": mean.view(-1), "rstd": rstd.view(-1)}
    rstd = s["rstd"][:, None]
    xhat = (x - s["mean"][:, None]) * rstd
    dy = s["dy"].float()
    d = dy * s["gamma"].float()
    dx = rstd * (d - d.mean(-1, keepdim=True) - xhat * (d * xhat).mean(-1, keepdim=True))
    return {"dx": dx.to(s["x"].dtype), "dgamma": (dy * xhat).sum(0), "dbeta": dy.sum(0)}


# ------------------------------------------------------------------ one pass
def run(state):
    if not own:
        return _plain(state)
    import bit_fwht_hadamard_b200 as q
    s, op = state, state["op"]
    if op == "gemm_epilogue":
        y, z = q.gemm_epilogue(s["A"], s["B"], s["M"], s["N"], s["K"], FMTS[s["fmt"]], bias=s["bias_t"],
                               act=ACTS[s["act"]], want_preact=s["preact"], dropout_p=s["p"], seed=s["seed"],
                               step=s["step"], residual=s["residual_t"], out_dtype=DTYPES[s["out"]])
        return {"y": y, "preact": z}
    if op == "epilogue_backward":
        dz, dbias = q.epilogue_backward(s["dy"], s["z"], act=ACTS[s["act"]], dropout_p=s["p"], seed=s["seed"],
                                        step=s["step"])
        return {"dz": dz, "dbias": dbias}
    if op == "dropout":
        return {"y": q.dropout(s["x"], s["p"], seed=s["seed"], step=s["step"], residual=s["residual_t"])}
    if op == "layernorm_forward":
        y, mean, rstd = q.layernorm_forward(s["x"], s["gamma"], s["beta"], eps=1e-5)
        return {"y": y, "mean": mean, "rstd": rstd}
    dx, dgamma, dbeta = q.layernorm_backward(s["dy"], s["x"], s["gamma"], s["mean"], s["rstd"])
    return {"dx": dx, "dgamma": dgamma, "dbeta": dbeta}


# ------------------------------------------------------------------ the definition in 64 bits
def _keep64(n, p, seed, step):
    """Which of elements 0 .. n-1 stay, from Philox's definition in 16-bit limbs (no product passes 2^34)."""
    q = torch.arange(-(-n // 4), device=DEV, dtype=torch.int64)
    ctr = [q % 2 ** 32, q // 2 ** 32, torch.full_like(q, step % 2 ** 32), torch.full_like(q, 2 ** 31 + step // 2 ** 32)]
    key = [seed % 2 ** 32, seed // 2 ** 32 % 2 ** 32]

    def mul(a, m):
        low, high = a % 65536 * m, a // 65536 * m            # a * m = low + 65536 * high, both below 2^48
        mid = low // 65536 + high                             # below 2^49
        return mid // 65536, mid % 65536 * 65536 + low % 65536

    for r in range(10):
        h0, l0 = mul(ctr[0], 0xD2511F53)
        h1, l1 = mul(ctr[2], 0xCD9E8D57)
        kk = [(key[0] + r * 0x9E3779B9) % 2 ** 32, (key[1] + r * 0xBB67AE85) % 2 ** 32]
        ctr = [h1 ^ ctr[1] ^ kk[0], l1, h0 ^ ctr[3] ^ kk[1], l0]
    words = torch.empty(4 * q.numel(), dtype=torch.int64, device=DEV)
    for j in range(4):
        words[j::4] = ctr[j]
    return words[:n].double() / 2.0 ** 32 >= int(p * 2.0 ** 32) / 2.0 ** 32


def _decode64(t, fmt):
    c, sc = t["codes"].long(), t["scales"].long()

    def e4m3(b):
        e, m = b // 8 % 16, (b % 8).double()
        v = torch.where(e == 0, m / 8 * 2.0 ** -6, (1 + m / 8) * torch.pow(2.0, (e - 7).double()))
        return torch.where(b >= 128, -v, v)

    if fmt == "mxfp8":
        v = e4m3(c)
    else:
        c = torch.cat([(c % 16)[..., None], (c // 16)[..., None]], -1).flatten(1)
        e, m = c // 2 % 4, (c % 2).double()
        v = torch.where(e == 0, m / 2, (1 + m / 2) * torch.pow(2.0, (e - 1).double()))
        v = torch.where(c >= 8, -v, v)
    s = e4m3(sc) if fmt == "nvfp4" else torch.pow(2.0, (sc - 127).double())
    if "tscale" in t:
        s = s * t["tscale"].double()
    return v * s.repeat_interleave(GROUP[fmt], 1)


def exact(case, seed):
    s = prepare(case, seed)
    op, p, step = case["op"], case.get("p", 0.0), int(s["step"])

    def drop(v):
        if p == 0.0:
            return v
        return v.mul_(_keep64(v.numel(), p, s["seed"], step).view(v.shape)).div_(1.0 - p)

    def cdf(z):
        return 0.5 * torch.special.erfc(-z / math.sqrt(2.0))

    def act(z):
        return {"none": lambda: z.clone(), "relu": lambda: z.clamp_min(0), "gelu": lambda: z * cdf(z),
                "gelu_tanh": lambda: z * torch.sigmoid(math.sqrt(8.0 / math.pi) * (z + 0.044715 * z ** 3)),
                "silu": lambda: z * torch.sigmoid(z)}[case["act"]]()

    def slope(z):
        if case["act"] == "gelu":
            return cdf(z) + z * torch.exp(-z * z / 2) / math.sqrt(2 * math.pi)
        if case["act"] == "gelu_tanh":
            f = torch.sigmoid(math.sqrt(8.0 / math.pi) * (z + 0.044715 * z ** 3))
            return f + z * f * (1 - f) * math.sqrt(8.0 / math.pi) * (1 + 0.134145 * z ** 2)
        if case["act"] == "silu":
            f = torch.sigmoid(z)
            return f + z * f * (1 - f)
        return (z > 0).double() if case["act"] == "relu" else torch.ones_like(z)

    if op == "gemm_epilogue":
        z = _decode64(s["A"], case["fmt"]) @ _decode64(s["B"], case["fmt"]).T
        if s["bias_t"] is not None:
            z = z + s["bias_t"].double()
        y = drop(act(z))
        if s["residual_t"] is not None:
            y = y + s["residual_t"].double()
        return {"y": y, "preact": z if case["preact"] else None}
    if op == "epilogue_backward":
        d = drop(s["dy"].double()) * slope(s["z"].double())
        return {"dz": d, "dbias": d.sum(0)}
    if op == "dropout":
        y = drop(s["x"].double())
        return {"y": y if s["residual_t"] is None else y + s["residual_t"].double()}
    x, gamma = s["x"].double(), s["gamma"].double()
    if op == "layernorm_forward":
        var, mean = torch.var_mean(x, -1, correction=0)
        rstd = (var + 1e-5) ** -0.5
        return {"y": (x - mean[:, None]) * rstd[:, None] * gamma + s["beta"].double(), "mean": mean, "rstd": rstd}
    dy, mean, rstd = s["dy"].double(), s["mean"].double()[:, None], s["rstd"].double()[:, None]
    n = (x - mean) * rstd
    d = dy * gamma
    dx = rstd * (d - d.mean(1, True) - n * (n * d).mean(1, True))
    return {"dx": dx, "dgamma": (dy * n).sum(0), "dbeta": dy.sum(0)}
