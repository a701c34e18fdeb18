"""The layer's row movement and its 4-bit experts, as cases to be measured.

Two families of operators that stand beside the dispatch, the grouped SwiGLU
and the combine:

* token rows sorted by expert (``permute_rows``) and back in token order with
  the routing weights applied (``unpermute_rows``), each with its gradient;
* microscaled 4-bit floating point (e2m1 values, one power-of-two scale for
  every 32): quantisation in token order or straight into sorted order, and the
  grouped products of 4-bit rows with 4-bit expert weights, the plain one
  (down) and the one that ends in SwiGLU (gate_up).

``own`` chooses between the plain form (elementary torch operations in fp32)
and the calls a user makes of ``sparse_top_mixture_b200``.
"""

import math

import torch

own = False

DTYPES = {"f32": torch.float32, "bf16": torch.bfloat16}


# ---- cases ------------------------------------------------------------------

def listed():
    return [
        # One decode batch of a 256-expert layer: its k expert rows summed back, where the launch is what counts.
        dict(name="unpermute decode", op="unpermute", T=16, H=7168, E=256, k=8, dtype="bf16", empty=0.0),
        # A training batch copied to its experts' segments.
        dict(name="permute train", op="permute", T=8192, H=4096, E=64, k=6, dtype="bf16", empty=0.0),
        # The gradient of that copy for the 128-expert top-8 layer: k rows summed per token.
        dict(name="permute grad train", op="permute_grad", T=4096, H=2048, E=128, k=8, dtype="bf16", empty=0.0),
        # The weighted return of a training batch.
        dict(name="unpermute train", op="unpermute", T=8192, H=4096, E=64, k=6, dtype="bf16", empty=0.0),
        # Its gradient, rows and routing weights, with the skew and the unused slots of an expert-parallel rank.
        dict(name="unpermute grad train", op="unpermute_grad", T=8192, H=2048, E=64, k=6, dtype="bf16", empty=0.25),
        # The same in fp32 for the small fp32 layer, an odd batch.
        dict(name="unpermute grad small f32", op="unpermute_grad", T=257, H=256, E=8, k=2, dtype="f32", empty=0.0),
        # Expert weights to 4 bits, as after loading or after a training step (16 experts' gate_up).
        dict(name="quantize weights", op="quantize", rows=16 * 2816, K=2048, dtype="bf16"),
        # A decode batch to 4 bits, straight into its experts' segments.
        dict(name="quantize sorted decode", op="quantize_sorted", T=16, H=7168, E=256, k=8, dtype="bf16", empty=0.0),
        # The down product of a decode batch that streams its experts' weights, in fp32 as the combine takes it.
        dict(name="product decode", op="product", T=16, E=256, k=8, N=7168, K=2048, out="f32"),
        # The down product of the 128-expert top-8 layer, a prefill batch.
        dict(name="product prefill", op="product", T=4096, E=128, k=8, N=2048, K=768, out="bf16"),
        # The gate_up product with its SwiGLU for one token, and for a large batch.
        dict(name="gate_up one token", op="gate_up", T=1, H=2048, E=128, k=8, I=768),
        dict(name="gate_up prefill", op="gate_up", T=8192, H=4096, E=64, k=6, I=2048),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(("permute", "permute_grad", "unpermute", "unpermute_grad", "quantize", "quantize_sorted", "product",
                     "gate_up"))
    E = rng.choice((4, 8, 16, 60, 64, 128, 160, 256))
    k = rng.randint(1, min(8, E))
    if op == "quantize":
        K = 32 * _log(rng, 1, 256)
        return dict(op=op, rows=_log(rng, 1, max(1, 16 * 2816 * 2048 // K)), K=K, dtype=rng.choice(("bf16", "f32")))
    if op == "product":
        N, K = 8 * _log(rng, 4, 896), 32 * _log(rng, 1, 224)
        most = max(1, min(4096, 4096 * 8 * 2048 * 768 // (k * N * K)))
        E = max(1, min(E, 128 * 2048 * 768 // (N * K)))
        return dict(op=op, T=_log(rng, 1, most), E=E, k=min(k, E), N=N, K=K, out=rng.choice(("bf16", "f32")))
    if op == "gate_up":
        H, I = 32 * _log(rng, 2, 224), 32 * _log(rng, 1, 64)
        most = max(1, min(8192, 8192 * 6 * 4096 * 2048 // (2 * k * H * I)))
        E = max(1, min(E, 64 * 4096 * 2048 // (H * I)))
        return dict(op=op, T=_log(rng, 1, most), H=H, E=E, k=min(k, E), I=I)
    unit = 32 if op == "quantize_sorted" else 8
    H = unit * _log(rng, 64 // unit, 7168 // unit)
    most = max(1, min(8192, 8192 * 6 * 4096 // (2 * k * H)))
    return dict(op=op, T=_log(rng, 1, most), H=H, E=E, k=k, dtype=rng.choice(("bf16", "bf16", "f32")),
                empty=rng.choice((0.0, 0.0, 0.3)))


# ---- inputs -----------------------------------------------------------------

def _generator(seed):
    return torch.Generator(device="cuda").manual_seed(int(seed))


def _randn(g, *shape, dtype=torch.float32, std=1.0):
    return (torch.randn(*shape, generator=g, device="cuda", dtype=torch.float32) * std).to(dtype)


def _plan(g, T, E, k, empty=0.0):
    """A top-k choice over unevenly liked experts, and its sorted segments: what the dispatch returns."""
    liking = _randn(g, E, std=0.5)
    noise = torch.rand(T, E, generator=g, device="cuda").clamp_(1e-6, 1 - 1e-6)
    selected = (liking - torch.log(-torch.log(noise))).topk(k, dim=1).indices
    scores = torch.rand(T, k, generator=g, device="cuda") + 0.1
    weights = scores / scores.sum(1, keepdim=True)
    if empty:  # slots without a row, as an expert-parallel rank has them
        selected = torch.where(torch.rand(T, k, generator=g, device="cuda") < empty, -1, selected)
    ids = selected.reshape(-1)
    P = ids.numel()
    order = torch.sort(torch.where(ids < 0, E, ids), stable=True).indices
    used = int((ids >= 0).sum())
    counts = torch.bincount(ids[ids >= 0], minlength=E)
    offsets = torch.zeros(E + 1, dtype=torch.int32, device="cuda")
    offsets[1:] = counts.cumsum(0)
    pair_pos = torch.full((P,), -1, dtype=torch.int32, device="cuda")
    pair_pos[order[:used]] = torch.arange(used, dtype=torch.int32, device="cuda")
    plan = {"counts": counts.to(torch.int32), "offsets": offsets, "sorted_pairs": order.to(torch.int32),
            "pair_pos": pair_pos}
    return plan, weights


def _weights4(g, E, N, K):
    """E experts' [N, K] weights of variance 1/K, in 4 bits."""
    data = torch.empty(E, N, K // 2, dtype=torch.uint8, device="cuda")
    scale = torch.empty(E, N, 16 * -(-K // 512), dtype=torch.uint8, device="cuda")
    for e in range(E):
        data[e], scale[e] = _quantize(_randn(g, N, K, dtype=torch.bfloat16, std=K ** -0.5))
    return data, scale


def _groups(s):
    """What the plain grouped product goes by: the experts that have rows, and their most rows."""
    counts = s["plan"]["counts"].long()
    s["active"] = counts.nonzero().reshape(-1)
    s["cap"] = int(counts.max())
    s["used"] = int(counts.sum())


def prepare(case, seed):
    c, g = case, _generator(seed)
    s = {"case": c}
    op = c["op"]
    if op == "quantize":
        s["x"] = _randn(g, c["rows"], c["K"], dtype=DTYPES[c["dtype"]], std=c["K"] ** -0.5)
        return s
    if op in ("product", "gate_up"):
        K, N = (c["K"], c["N"]) if op == "product" else (c["H"], 2 * c["I"])
        s["plan"], _ = _plan(g, c["T"], c["E"], c["k"])
        s["a"] = _quantize(_randn(g, c["T"] * c["k"], K, dtype=torch.bfloat16))
        s["w"] = _weights4(g, c["E"], N, K)
        _groups(s)
        return s
    dt = DTYPES[c["dtype"]]
    s["plan"], s["weights"] = _plan(g, c["T"], c["E"], c["k"], c["empty"])
    if op in ("permute", "quantize_sorted"):
        s["x"] = _randn(g, c["T"], c["H"], dtype=dt)
    elif op == "permute_grad":
        s["dx_perm"] = _randn(g, c["T"] * c["k"], c["H"], dtype=dt)
    else:
        s["y_perm"] = _randn(g, c["T"] * c["k"], c["H"], dtype=dt)
        if op == "unpermute_grad":
            s["dout"] = _randn(g, c["T"], c["H"], dtype=dt)
    return s


# ---- the plain forms --------------------------------------------------------

def _pow2(byte):
    """2^(byte - 127) in fp32, exactly, for 1 <= byte <= 254 (0, the scale of a block of zeros, gives 0)."""
    return (byte.to(torch.int32) << 23).view(torch.float32)


def _quantize(x):
    """4-bit values, two to a byte (the even one low), and the scale bytes, padded with zeros to 16."""
    rows, K = x.shape
    v = x.float().reshape(rows, K // 32, 32)
    top = torch.frexp(v.abs().amax(2)).exponent - 1  # floor(log2(largest))
    byte = (top + 125).clamp(0, 254)
    byte = torch.where(v.abs().amax(2) > 0, byte, 0)
    a = v * _pow2(254 - byte)[:, :, None]
    m = a.abs()
    code = ((m > 0.25).to(torch.uint8) + (m >= 0.75) + (m > 1.25) + (m >= 1.75) + (m > 2.5) + (m >= 3.5) + (m > 5.0))
    code = (code + 8 * torch.signbit(a)).to(torch.uint8).reshape(rows, K // 2, 2)
    scale = torch.zeros(rows, 16 * -(-K // 512), dtype=torch.uint8, device=x.device)
    scale[:, : K // 32] = byte.to(torch.uint8)
    return code[:, :, 0] + 16 * code[:, :, 1], scale


def _values(data, scale):
    """The fp32 values of 4-bit rows [..., K/2] with scale bytes [..., S]."""
    e2m1 = torch.tensor([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0, -0.0, -0.5, -1.0, -1.5, -2.0, -3.0, -4.0, -6.0],
                        device=data.device)
    v = torch.stack((e2m1[(data & 15).int()], e2m1[(data >> 4).int()]), -1)
    n = data.shape[-1] // 16
    return (v.reshape(*data.shape[:-1], n, 32) * _pow2(scale[..., :n])[..., None]).flatten(-2)


def _grouped(s, a, w):
    """a [P, K] times each row's expert's w [E, N, K], in fp32: the experts' rows padded to the most of one."""
    off = s["plan"]["offsets"].long()
    act, cap, used = s["active"], s["cap"], s["used"]
    at = (off[act][:, None] + torch.arange(cap, device=a.device)).clamp(max=a.shape[0] - 1)
    y = torch.bmm(a[at], _values(w[0][act], w[1][act]).transpose(1, 2))
    rows = torch.arange(used, device=a.device)
    e = torch.searchsorted(off[act] + s["plan"]["counts"].long()[act], rows, right=True)
    return y[e, rows - off[act][e]]


def _plain(s):
    c, op = s["case"], s["case"]["op"]
    if op == "quantize":
        return _values(*_quantize(s["x"])).to(torch.bfloat16)
    if op == "product":
        return _grouped(s, _values(*s["a"]), s["w"]).to(DTYPES[c["out"]])
    if op == "gate_up":
        gate, up = _grouped(s, _values(*s["a"]), s["w"]).chunk(2, 1)
        return (gate / (1 + torch.exp(-gate)) * up).to(torch.bfloat16)
    plan, T, k = s["plan"], c["T"], c["k"]
    pos = plan["pair_pos"].long().reshape(T, k)
    has, at = (pos >= 0)[:, :, None], pos.clamp(min=0)
    token = plan["sorted_pairs"].long() // k
    filled = (torch.arange(T * k, device="cuda") < plan["offsets"][-1])[:, None]
    if op == "permute":
        return torch.where(filled, s["x"][token], 0)
    if op == "quantize_sorted":
        rows = torch.where(filled, s["x"][token], 0)
        return _values(*_quantize(rows)).to(torch.bfloat16)
    if op == "permute_grad":
        return torch.where(has, s["dx_perm"][at].float(), 0).sum(1).to(s["dx_perm"].dtype)
    y = torch.where(has, s["y_perm"][at].float(), 0)
    if op == "unpermute":
        return (y * s["weights"][:, :, None]).sum(1).to(s["y_perm"].dtype)
    dout = s["dout"].float()
    pair = plan["sorted_pairs"].long()
    dy = torch.where(filled, dout[token] * s["weights"].reshape(-1)[pair][:, None], 0).to(s["y_perm"].dtype)
    return {"dy_perm": dy, "d_weights": (y * dout[:, None]).sum(2)}


# ---- the framework's calls --------------------------------------------------

def _own(s):
    import sparse_top_mixture_b200 as stm

    c, op = s["case"], s["case"]["op"]
    if op == "quantize":
        return stm.mx4_dequantize(stm.mx4_quantize(s["x"]))
    if op == "product":
        return stm.mx4_grouped_matmul(stm.Mx4(*s["a"]), stm.Mx4(*s["w"]), s["plan"]["offsets"], DTYPES[c["out"]])
    if op == "gate_up":
        return stm.mx4_grouped_gate_up(stm.Mx4(*s["a"]), stm.Mx4(*s["w"]), s["plan"]["offsets"])
    p = stm.Problem(T=c["T"], H=c["H"], E=c["E"], k=c["k"], I=8, dtype=c["dtype"])
    if op == "permute":
        return stm.permute_rows(p, s["x"], s["plan"])
    if op == "quantize_sorted":
        return stm.mx4_dequantize(stm.mx4_permute_rows(p, s["x"], s["plan"]))
    if op == "permute_grad":
        return stm.permute_rows_backward(p, s["dx_perm"], s["plan"])
    if op == "unpermute":
        return stm.unpermute_rows(p, s["y_perm"], s["plan"], s["weights"])
    dy, dw = stm.unpermute_rows_backward(p, s["dout"], s["y_perm"], s["plan"], s["weights"])
    return {"dy_perm": dy, "d_weights": dw}


def run(state):
    return _own(state) if own else _plain(state)


# ---- what a pass cannot do without ------------------------------------------

def work(case):
    c, op = case, case["op"]
    four = lambda n: n * (0.5 + 1 / 32)  # noqa: E731  bytes of n 4-bit values and their scales
    if op == "quantize":
        n, es = c["rows"] * c["K"], 2 if c["dtype"] == "bf16" else 4
        return {"bytes": n * (es + 2) + four(n), "flops": 0}
    T, k, E = c["T"], c["k"], c["E"]
    P = T * k
    touched = E * (1 - (1 - k / E) ** T)  # experts that some token chose
    if op == "product":
        out = 2 if c["out"] == "bf16" else 4
        return {"bytes": four(P * c["K"]) + four(touched * c["N"] * c["K"]) + P * c["N"] * out,
                "flops": 2 * P * c["N"] * c["K"]}
    if op == "gate_up":
        return {"bytes": four(P * c["H"]) + four(touched * 2 * c["I"] * c["H"]) + P * c["I"] * 2,
                "flops": 4 * P * c["I"] * c["H"]}
    es = 2 if c["dtype"] == "bf16" else 4
    rows, H = P * (1 - c["empty"]), c["H"]
    if op in ("permute", "permute_grad"):
        return {"bytes": (T + P) * H * es + 4 * P, "flops": 0}
    if op == "quantize_sorted":
        return {"bytes": T * H * es + four(P * H) + P * H * 2 + 4 * P, "flops": 0}
    if op == "unpermute":
        return {"bytes": (T + rows) * H * es + 8 * P, "flops": 2 * rows * H}
    return {"bytes": (T + rows + P) * H * es + 12 * P, "flops": 3 * rows * H}


# ---- the definitions in 64 bits ---------------------------------------------

_GRID = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)


def _exact_pow2(n):
    """2^n in 64 bits for whole n, by its exponent field (the device's pow is not exact)."""
    return ((n.long() + 1023) << 52).view(torch.float64)


def _exact_quantized(x):
    """Each value's nearest of _GRID times the block's power of two (a tie: the one of even index), in 64 bits."""
    rows, K = x.shape
    b = x.double().reshape(-1, 32)
    largest = b.abs().max(1, keepdim=True).values
    power = torch.floor(torch.log2(largest.clamp(min=2.0 ** -140)))
    power += (_exact_pow2(power + 1) <= largest).double() - (_exact_pow2(power) > largest).double()
    unit = _exact_pow2((power - 2).clamp(-127, 127))
    a = b.abs() / unit
    best, far = torch.zeros_like(a), a.clone()
    for i, v in enumerate(_GRID[1:], 1):
        d = (a - v).abs()
        take = (d < far) | ((d == far) & (i % 2 == 0))
        best, far = torch.where(take, v, best), torch.where(take, d, far)
    return (torch.sign(b) * best * unit).reshape(rows, K)


def _exact_values(data, scale):
    n = data.shape[-1] * 2
    nib = torch.empty(*data.shape[:-1], n, dtype=torch.long, device=data.device)
    nib[..., 0::2], nib[..., 1::2] = data % 16, data // 16
    v = torch.tensor(_GRID, dtype=torch.float64, device=data.device)[nib % 8] * torch.where(nib >= 8, -1.0, 1.0).double()
    return v * torch.repeat_interleave(_exact_pow2(scale.long() - 127), 32, dim=-1)[..., :n]


def exact(case, seed):
    s = prepare(case, seed)
    c, op = case, case["op"]
    if op == "quantize":
        return torch.cat([_exact_quantized(r) for r in s["x"].split(4096)])
    offsets = s["plan"]["offsets"].tolist()
    if op in ("product", "gate_up"):
        y = []
        for e in range(c["E"]):
            lo, hi = offsets[e], offsets[e + 1]
            if hi > lo:
                y.append(_exact_values(s["a"][0][lo:hi], s["a"][1][lo:hi]) @ _exact_values(s["w"][0][e], s["w"][1][e]).T)
        y = torch.cat(y)
        return y if op == "product" else y[:, : c["I"]] * torch.sigmoid(y[:, : c["I"]]) * y[:, c["I"]:]
    T, k, H = c["T"], c["k"], c["H"]
    pos = s["plan"]["pair_pos"].long()
    pairs = (pos >= 0).nonzero().reshape(-1)
    if op in ("permute", "quantize_sorted"):
        rows = torch.zeros(T * k, H, dtype=torch.float64, device="cuda")
        x = s["x"].double() if op == "permute" else _exact_quantized(s["x"])
        rows[pos[pairs]] = x[pairs // k]
        return rows
    if op == "permute_grad":
        return torch.zeros(T, H, dtype=torch.float64, device="cuda").index_add_(0, pairs // k, s["dx_perm"].double()[pos[pairs]])
    w = s["weights"].double().reshape(-1)
    if op == "unpermute":
        rows = s["y_perm"].double()[pos[pairs]] * w[pairs][:, None]
        return torch.zeros(T, H, dtype=torch.float64, device="cuda").index_add_(0, pairs // k, rows)
    dy = torch.zeros(T * k, H, dtype=torch.float64, device="cuda")
    dw = torch.zeros(T * k, dtype=torch.float64, device="cuda")
    for some in pairs.split(4096):
        d = s["dout"].double()[some // k]
        dy[pos[some]] = d * w[some][:, None]
        dw[some] = (d * s["y_perm"].double()[pos[some]]).sum(1)
    return {"dy_perm": dy, "d_weights": dw.reshape(T, k)}
