"""Measured cases of the microscaled (MX) products, the MX quantisation and the RMS norms.

``own`` false: the operators in elementary torch operations.  ``own`` true: the calls a user
makes of this package.  Activations and weights follow the shapes this library is measured
on: hidden size 5120, projections of 12288 and 17408 rows, 6144- and 17408-column inputs, one
to 64 tokens in decode and verification, 1024 to 4096 in prefill.

MX block: 32 consecutive values share one power-of-two scale 2^E, E = floor(log2 max|v|) - emax;
elements are E2M1 (emax 2, largest 6) or E4M3 (emax 8, largest 448), rounded to nearest even.
"""
import math

import torch

own = False

EPS = 1e-6
DTYPES = {"fp16": torch.float16, "bf16": torch.bfloat16}


def listed():
    return [
        # one decode token's hidden state, to 4 bits and back: launch latency
        {"name": "quantize_decode", "op": "quantize", "T": 1, "K": 5120, "fmt": 4, "dtype": "fp16"},
        # the down projection's input of a long prompt, to 4 bits and back
        {"name": "quantize_prefill", "op": "quantize", "T": 4096, "K": 17408, "fmt": 4, "dtype": "bf16"},
        # the norm before a decode step's projections, with the residual's addition
        {"name": "norm_decode", "op": "norm", "T": 1, "K": 5120, "out": "16", "residual": True, "dtype": "fp16"},
        # an odd width and a token count between powers of two, no residual (the first layer's norm)
        {"name": "norm_odd", "op": "norm", "T": 777, "K": 5119, "out": "16", "residual": False, "dtype": "bf16"},
        # the norm of a prompt chunk in front of the int8-activation products
        {"name": "norm_a8", "op": "norm", "T": 1024, "K": 5120, "out": "a8", "residual": True, "dtype": "fp16"},
        # the norm of a long prompt in front of the MX products
        {"name": "norm_mx_prefill", "op": "norm", "T": 4096, "K": 5120, "out": "mx8", "residual": True, "dtype": "bf16"},
        # the smallest product: latency alone
        {"name": "linear_tiny", "op": "linear", "T": 1, "N": 256, "K": 512, "fmt": 8, "dtype": "fp16"},
        # a verification of four tokens: bound by the weights' bytes
        {"name": "linear_verify", "op": "linear", "T": 4, "N": 12288, "K": 5120, "fmt": 8, "dtype": "fp16"},
        # the gate/up pair at a wide batch of decode tokens
        {"name": "swiglu_batch", "op": "swiglu", "T": 64, "N": 17408, "K": 5120, "fmt": 8, "dtype": "bf16"},
        # the gate/up pair of a prompt chunk, activations in 4 bits too
        {"name": "swiglu_prefill", "op": "swiglu", "T": 1024, "N": 17408, "K": 5120, "fmt": 4, "dtype": "fp16"},
        # the down projection of two decode tokens: few rows, long sums
        {"name": "add_decode", "op": "add", "T": 2, "N": 5120, "K": 17408, "fmt": 4, "dtype": "bf16"},
        # the output projection of a long prompt with the residual's addition
        {"name": "add_prefill", "op": "add", "T": 4096, "N": 5120, "K": 6144, "fmt": 4, "dtype": "fp16"},
    ]


def _log(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["quantize", "norm", "linear", "swiglu", "add"])
    case = {"op": op, "T": _log(rng, 1, 4096), "dtype": rng.choice(["fp16", "bf16"])}
    if op == "quantize":
        return case | {"K": 32 * _log(rng, 1, 544), "fmt": rng.choice([4, 8])}
    if op == "norm":
        out = rng.choice(["16", "a8", "mx8"])
        K = {"16": 1, "a8": 64, "mx8": 32}[out]
        return case | {"K": K * _log(rng, 64 // K, 17408 // K), "out": out, "residual": rng.random() < 0.7}
    N, K = 16 * _log(rng, 4, 1088), 32 * _log(rng, 4, 544)
    rows = 2 * N if op == "swiglu" else N
    T = max(1, min(case["T"], 1024 * 2 * 17408 * 5120 // (rows * K)))
    return case | {"T": T, "N": N, "K": K, "fmt": rng.choice([4, 8])}


# ---- elementary forms

def _mx_plain(v, fmt):
    """fp32 v [R, K] -> (element values fp32 [R, K], exponents int32 [R, K/32])."""
    emax, emin, man, top = (2, 0, 1, 6.0) if fmt == 4 else (8, -6, 3, 448.0)
    b = v.reshape(v.shape[0], -1, 32)
    m = b.abs().amax(-1, keepdim=True)
    e = torch.frexp(m).exponent - 1 - emax
    e = torch.where(m == 0, -127, e.clamp(-127, 127))
    s = torch.ldexp(b, -e)
    step = (torch.frexp(s).exponent - 1).clamp(min=emin) - man  # the spacing of the values near s
    q = torch.ldexp(torch.round(torch.ldexp(s, -step)), step).clamp(-top, top)
    return q.reshape(v.shape), e.squeeze(-1)


def _mx_value(q, e):
    return torch.ldexp(q.reshape(q.shape[0], -1, 32), e.unsqueeze(-1)).reshape(q.shape)


def _e2m1_codes(q):
    """Element values -> codes, two to a byte, the even column in the low half."""
    a = q.abs()
    code = torch.where(a < 2, a * 2, torch.where(a < 4, a + 2, a / 2 + 4)).to(torch.uint8)
    code = code | (torch.signbit(q).to(torch.uint8) << 3)
    return code[:, ::2] | (code[:, 1::2] << 4)


def _weight_plain(codes, scales):
    """Codes uint8 [N, K/2], scale bytes uint8 [N, K/32] -> fp32 [N, K]."""
    table = torch.tensor([0, 0.5, 1, 1.5, 2, 3, 4, 6, 0, -0.5, -1, -1.5, -2, -3, -4, -6], device=codes.device)
    idx = torch.stack([codes & 15, codes >> 4], -1).reshape(codes.shape[0], -1)
    return _mx_value(table[idx.int()], scales.int() - 127)


def _norm_plain(x, r, w):
    h = x.float() if r is None else x.float() + r.float()
    rstd = torch.rsqrt(h.double().square().mean(-1, keepdim=True) + EPS).float()
    return h, h * rstd * w.float()


def _a8_value(y):
    """y [T, K] through int8 with a scale per 64 columns and back."""
    g = y.reshape(y.shape[0], -1, 64)
    s = g.abs().amax(-1, keepdim=True) / 127
    q = torch.where(s > 0, torch.round(g / s), 0).clamp(-127, 127)
    return (q * s).reshape(y.shape)


# ---- the cases

def _normal(g, *shape):
    return torch.randn(*shape, generator=g, device="cuda")


def _activations(g, T, K, dtype):
    """N(0, 1) with a few channels thirty times as large, as projections' inputs have."""
    x = _normal(g, T, K)
    x[:, torch.randint(K, (max(1, K // 640),), generator=g, device="cuda")] *= 30
    return x.to(dtype)


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    s, dtype = dict(case), DTYPES[case["dtype"]]
    T, K, op = case["T"], case["K"], case["op"]
    s["x"] = _activations(g, T, K, dtype)
    if op == "norm":
        s["r"] = _normal(g, T, K).to(dtype) if case["residual"] else None
        s["w"] = (1 + 0.1 * _normal(g, K)).to(dtype)
    if op in ("linear", "swiglu", "add"):
        N = case["N"]
        s["weights"] = []
        for _ in range(2 if op == "swiglu" else 1):
            q, e = _mx_plain(0.02 * _normal(g, N, K), 4)
            s["weights"].append((_e2m1_codes(q), (e + 127).to(torch.uint8)))
        if op == "add":
            s["r"] = _normal(g, T, N).to(dtype)
    if own:
        import w4_groupwise_gemm_amd as w4
        if op == "swiglu":
            s["pw"] = w4.pack_mx_pair(*s["weights"], device="cuda")
        elif op in ("linear", "add"):
            s["pw"] = w4.pack_mx(*s["weights"][0], device="cuda")
    return s


def _run_own(s):
    import w4_groupwise_gemm_amd as w4
    op = s["op"]
    if op == "quantize":
        return w4.dequantize_mx(w4.quantize_mx(s["x"], fmt=s["fmt"]), dtype=torch.bfloat16)
    if op == "norm":
        if s["out"] == "16":
            y, h = w4.rmsnorm(s["x"], s["w"], eps=EPS, residual=s["r"])
        elif s["out"] == "a8":
            ws, h = w4.rmsnorm_a8(s["x"], s["w"], eps=EPS, residual=s["r"])
            y = w4.dequantize_a8(ws, s["T"], s["K"], dtype=s["x"].dtype)
        else:
            q, h = w4.rmsnorm_mx(s["x"], s["w"], fmt=8, eps=EPS, residual=s["r"])
            y = [q.codes.view(torch.float8_e4m3fn), q.scales.view(torch.float8_e8m0fnu)]
        return [y] if h is None else [y, h]
    if op == "linear":
        return w4.linear_mx(s["x"], s["pw"], fmt=s["fmt"])
    if op == "swiglu":
        return w4.linear_swiglu_mx(s["x"], s["pw"], fmt=s["fmt"])
    return w4.linear_add_mx(s["x"], s["pw"], s["r"], fmt=s["fmt"])


def run(s):
    if own:
        return _run_own(s)
    op, x = s["op"], s["x"]
    if op == "quantize":
        return _mx_value(*_mx_plain(x.float(), s["fmt"])).to(torch.bfloat16)
    if op == "norm":
        h, y = _norm_plain(x, s["r"], s["w"])
        if s["out"] == "16":
            y = y.to(x.dtype)
        elif s["out"] == "a8":
            y = _a8_value(y).to(x.dtype)
        else:
            q, e = _mx_plain(y, 8)
            y = [q.to(torch.float8_e4m3fn), (e + 127).to(torch.uint8).view(torch.float8_e8m0fnu)]
        return [y] if s["r"] is None else [y, h.to(x.dtype)]
    a = _mx_value(*_mx_plain(x.float(), s["fmt"]))
    p = [a @ _weight_plain(*w).t() for w in s["weights"]]
    if op == "linear":
        y = p[0]
    elif op == "swiglu":
        y = p[0] / (1 + torch.exp(-p[0])) * p[1]
    else:
        y = p[0] + s["r"].float()
    return y.to(x.dtype)


def work(case):
    """Every input read once and every output written once; a product's multiplications and additions."""
    T, K, op = case["T"], case["K"], case["op"]
    if op == "quantize":
        code = T * K * case["fmt"] / 8 + T * K / 32
        return {"bytes": int(4 * T * K + 2 * code), "flops": 0}
    if op == "norm":
        out = {"16": 2, "a8": 1 + 4 / 64, "mx8": 1 + 1 / 32}[case["out"]] * T * K
        back = out + 2 * T * K if case["out"] == "a8" else 0  # read back to 16 bits
        return {"bytes": int((6 if case["residual"] else 2) * T * K + out + back + 2 * K), "flops": 0}
    N = case["N"]
    rows = 2 * N if op == "swiglu" else N
    return {"bytes": int(rows * K * (0.5 + 1 / 32) + 2 * T * K + (4 if op == "add" else 2) * T * N), "flops": 2 * T * rows * K}


# ---- the definitions in 64 bits

def _grid(fmt):
    """The non-negative values of the element type, in order, as its exponent and mantissa fields give them."""
    man, bias, last = (1, 1, 7) if fmt == 4 else (3, 7, 126)
    vals = []
    for c in range(last + 1):
        e, m = c >> man, c & ((1 << man) - 1)
        vals.append(math.ldexp(m, 1 - bias - man) if e == 0 else math.ldexp((1 << man) + m, e - bias - man))
    return torch.tensor(vals, dtype=torch.float64, device="cuda")


def _mx_exact(v, fmt):
    """fp64 v [R, K] -> (elements, scales) in fp64: the nearest value of the grid, the even code on a tie."""
    grid = _grid(fmt)
    mid = (grid[1:] + grid[:-1]) / 2
    b = v.reshape(-1, 32)
    m = b.abs().max(1).values
    e = torch.floor(torch.log2(m))
    e = torch.where(torch.exp2(e) > m, e - 1, torch.where(torch.exp2(e + 1) <= m, e + 1, e))
    scale = torch.exp2((e - (2 if fmt == 4 else 8)).clamp(-127, 127))
    a = b.abs() / scale[:, None]
    i = torch.searchsorted(mid, a)
    i += (i % 2 == 1) & (i < len(mid)) & (a == mid[i.clamp(max=len(mid) - 1)])
    return (grid[i] * torch.sign(b)).reshape(v.shape), scale.reshape(v.shape[0], -1)


def exact(case, seed):
    s = prepare(case, seed)
    op, x = s["op"], s["x"].double()
    if op == "quantize":
        q, scale = _mx_exact(x, s["fmt"])
        return q * scale.repeat_interleave(32, 1)
    if op == "norm":
        h = x if s["r"] is None else x + s["r"].double()
        y = h / torch.sqrt((h * h).sum(1, keepdim=True) / s["K"] + EPS) * s["w"].double()
        if s["out"] == "a8":
            a = y.reshape(s["T"], -1, 64)
            unit = a.abs().max(2, keepdim=True).values / 127
            y = (torch.round(a / unit) * unit).reshape(y.shape)
        elif s["out"] == "mx8":
            y = list(_mx_exact(y, 8))
        return [y] if s["r"] is None else [y, h]
    q, scale = _mx_exact(x, s["fmt"])
    a = q * scale.repeat_interleave(32, 1)
    p = []
    for codes, bytes_ in s["weights"]:
        c = torch.empty(codes.shape[0], s["K"], dtype=torch.long, device="cuda")
        c[:, 0::2], c[:, 1::2] = codes % 16, codes // 16
        w = _grid(4)[c % 8] * (1 - 2 * (c // 8))
        p.append(a @ (w * torch.exp2(bytes_.double() - 127).repeat_interleave(32, 1)).t())
    if op == "linear":
        return p[0]
    if op == "swiglu":
        return p[0] * torch.sigmoid(p[0]) * p[1]
    return p[0] + s["r"].double()
