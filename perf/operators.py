"""The 8-bit operators of the per-token FFN, as cases that can be measured.

Four operators over sample-major activations [B, T, cols] (one weight matrix per token t):

  act8    a checkpoint in 8 bits: save (quantise) and restore
  matmul  the product of 8-bit activations with a token's 8-bit weights (both directions)
  wgrad   a weight's and a bias's gradient from an activation kept in 8 bits
  pffn    the two-layer per-token FFN on 8-bit operands: serving, and a training step that keeps
          its activations in 8 bits and runs backward from them

The 8-bit format: codes of 8 bits (e4m3, or e5m2) and one exponent byte E for every 128
consecutive values of a row (every 128 x 128 values of a weight); a value is code * 2^(E - 127).
E is the smallest that brings the block's largest finite value to at most the format's largest;
a block of zeros has E = 127.  Code rows are padded to a multiple of 16 bytes, exponent rows to a
multiple of 4.
"""
from __future__ import annotations

import math

import torch

own = False

FORMATS = {"e4m3": (torch.float8_e4m3fn, 9), "e5m2": (torch.float8_e5m2, 16)}   # largest = 0.875 * 2^top
DTYPES = {"bf16": torch.bfloat16, "f32": torch.float32}
BLOCK = 128


def listed() -> list[dict]:
    return [
        # one request's activations, kept and read back: the launch and its latency
        {"name": "act8 one sample", "op": "act8", "B": 1, "T": 32, "C": 1536, "dtype": "bf16", "fmt": "e4m3"},
        # a training batch's hidden activations of the 1B shape
        {"name": "act8 hidden 1B", "op": "act8", "B": 2048, "T": 32, "C": 6144, "dtype": "bf16", "fmt": "e4m3"},
        # float32 gradients of an odd shape, blocks that end inside the row
        {"name": "act8 odd f32 e5m2", "op": "act8", "B": 1237, "T": 5, "C": 1003, "dtype": "f32", "fmt": "e5m2"},
        # serving one request: weights streamed once
        {"name": "matmul one sample", "op": "matmul", "B": 1, "T": 32, "K": 1536, "N": 6144, "trans": False,
         "fmt": "e4m3", "bias": True},
        # a small serving batch against the second layer
        {"name": "matmul B64", "op": "matmul", "B": 64, "T": 32, "K": 6144, "N": 1536, "trans": False, "fmt": "e4m3",
         "bias": True},
        # a gradient in e5m2 against the transposed weights, nothing a multiple of a tile
        {"name": "matmul odd transposed", "op": "matmul", "B": 333, "T": 7, "K": 1000, "N": 713, "trans": True,
         "fmt": "e5m2", "bias": False},
        # the first layer at the batch of the 1B benchmark
        {"name": "matmul 1B", "op": "matmul", "B": 4096, "T": 32, "K": 1536, "N": 6144, "trans": False, "fmt": "e4m3",
         "bias": True},
        # the weight gradients of a small and of a large layer
        {"name": "wgrad odd", "op": "wgrad", "B": 777, "T": 6, "K": 528, "N": 1040},
        {"name": "wgrad 1B", "op": "wgrad", "B": 2048, "T": 32, "K": 1536, "N": 6144},
        # serving a handful of requests through the whole FFN
        {"name": "pffn serving B8", "op": "pffn", "B": 8, "T": 32, "D": 1536, "F": 6144, "train": False},
        # a training step of a small model, and of the 1B shape
        {"name": "pffn train small", "op": "pffn", "B": 250, "T": 8, "D": 512, "F": 2048, "train": True},
        {"name": "pffn train 1B", "op": "pffn", "B": 1024, "T": 32, "D": 1536, "F": 6144, "train": True},
    ]


def _log(rng, lo: int, hi: int, step: int = 1) -> int:
    v = math.exp(rng.uniform(math.log(lo), math.log(hi + step)))
    return max(lo, min(hi, int(v) // step * step))


def draw(rng) -> dict:
    """One more case: sizes spread over their logarithm, no more work than the largest listed of its kind."""
    op = rng.choice(["act8", "matmul", "wgrad", "pffn", "matmul", "pffn"])
    while True:
        B, T = _log(rng, 1, 4096), rng.randint(1, 40)
        if op == "act8":
            C = _log(rng, 1, 6144)
            if B * T * C <= 2048 * 32 * 6144:
                return {"op": op, "B": B, "T": T, "C": C, "dtype": rng.choice(["bf16", "f32"]),
                        "fmt": rng.choice(["e4m3", "e5m2"])}
        elif op == "matmul":
            K, N = _log(rng, 16, 6144), _log(rng, 16, 6144)
            if B * T * K * N <= 2048 * 32 * 1536 * 6144:
                return {"op": op, "B": B, "T": T, "K": K, "N": N, "trans": rng.random() < 0.5,
                        "fmt": rng.choice(["e4m3", "e4m3", "e5m2"]), "bias": rng.random() < 0.5}
        elif op == "wgrad":
            K, N = _log(rng, 16, 2048, 16), _log(rng, 16, 6144, 16)
            if B * T * K * N <= 1024 * 32 * 1536 * 6144:
                return {"op": op, "B": B, "T": T, "K": K, "N": N}
        else:
            D = _log(rng, 16, 2048, 16)
            F = D * rng.randint(1, 4)
            if B * T * D * F <= 512 * 32 * 1536 * 6144:
                return {"op": op, "B": B, "T": T, "D": D, "F": F, "train": rng.random() < 0.6}


# ---- the 8-bit format in elementary torch operations -------------------------------------------

def _pow2(e: torch.Tensor) -> torch.Tensor:
    """2^e in float32 for whole e in [-126, 127], exactly."""
    return ((e.to(torch.int32) + 127) << 23).view(torch.float32)


def _exponent(amax: torch.Tensor, top: int) -> torch.Tensor:
    """The smallest e with amax <= 0.875 * 2^(top + e); 0 for amax = 0; at least -126."""
    m, ex = torch.frexp(amax)
    e = (ex - top + (m > 0.875).to(ex.dtype)).clamp(min=-126)
    return torch.where(amax > 0, e, torch.zeros_like(e))


def _blocks(x: torch.Tensor, dim: int) -> torch.Tensor:
    """x padded with zeros along dim to whole blocks of 128 and cut into them: [.., blocks, 128, ..]."""
    dim %= x.dim()
    n = x.shape[dim]
    nb = -(-n // BLOCK)
    if nb * BLOCK != n:
        pad = [0, 0] * (x.dim() - 1 - dim) + [0, nb * BLOCK - n]
        x = torch.nn.functional.pad(x, pad)
    return x.reshape(x.shape[:dim] + (nb, BLOCK) + x.shape[dim + 1:])


def _quantise(x: torch.Tensor, fmt: str) -> tuple[torch.Tensor, torch.Tensor]:
    """(codes [.., blocks, 128], exponents [.., blocks]) of float32 rows."""
    f8, top = FORMATS[fmt]
    x = _blocks(x, -1)
    fine = torch.isfinite(x)
    e = _exponent(torch.where(fine, x.abs(), 0.0).amax(-1), top)
    return torch.where(fine, x * _pow2(-e).unsqueeze(-1), torch.nan).to(f8), e


def _restore(codes: torch.Tensor, e: torch.Tensor, cols: int) -> torch.Tensor:
    """float32 rows of cols values."""
    return (codes.float() * _pow2(e).unsqueeze(-1)).flatten(-2)[..., :cols]


def _rounded(x: torch.Tensor, fmt: str = "e4m3") -> torch.Tensor:
    """x as its 8-bit form stands for it."""
    return _restore(*_quantise(x, fmt), x.shape[-1])


def _stored(codes: torch.Tensor, e: torch.Tensor, cols: int) -> tuple[torch.Tensor, torch.Tensor]:
    """The layout in memory: code rows of a multiple of 16 bytes, exponent bytes E = e + 127 in rows of a multiple of 4."""
    ld, lds = -(-cols // 16) * 16, -(-e.shape[-1] // 4) * 4
    q = torch.zeros(e.shape[:-1] + (ld,), dtype=torch.uint8, device=e.device)
    q[..., :cols] = codes.view(torch.uint8).flatten(-2)[..., :cols]
    s = torch.full(e.shape[:-1] + (lds,), 127, dtype=torch.uint8, device=e.device)
    s[..., :e.shape[-1]] = (e + 127).to(torch.uint8)
    return q.view(codes.dtype), s


def _activation(B: int, T: int, C: int, g: torch.Generator) -> torch.Tensor:
    """Rows as they leave a LayerNorm with a learned affine: unit size, a few columns much larger, rows of differing size."""
    x = torch.randn((B, T, C), generator=g, device="cuda")
    x *= torch.exp(0.5 * torch.randn((B, T, 1), generator=g, device="cuda"))
    big = torch.rand((1, T, C), generator=g, device="cuda") < 0.002
    return torch.where(big, 20.0 * x, x)


def _act8(x: torch.Tensor, fmt: str = "e4m3") -> dict:
    codes, e = _quantise(x, fmt)
    q, s = _stored(codes, e, x.shape[-1])
    return {"q": q, "s": s, "cols": x.shape[-1]}


def _weight8(T: int, K: int, N: int, g: torch.Generator) -> dict:
    """A token-wise weight [T, K, N] ~ N(0, 1/K) in 8 bits: one exponent per 128 x 128 block."""
    q = torch.zeros((T, K, -(-N // 16) * 16), dtype=torch.float8_e4m3fn, device="cuda")
    kb, nb = -(-K // BLOCK), -(-N // BLOCK)
    s = torch.full((T, kb, -(-nb // 4) * 4), 127, dtype=torch.uint8, device="cuda")
    for t in range(T):
        w = torch.randn((K, N), generator=g, device="cuda") / math.sqrt(K)
        blocks = _blocks(_blocks(w, 1), 0)                        # [kb, 128, nb, 128]
        e = _exponent(blocks.abs().amax((1, 3)), 9)
        codes = (blocks * _pow2(-e)[:, None, :, None]).to(torch.float8_e4m3fn).view(torch.uint8)
        q[t].view(torch.uint8)[:, :N] = codes.reshape(kb * BLOCK, nb * BLOCK)[:K, :N]
        s[t, :, :nb] = (e + 127).to(torch.uint8)
    return {"q": q, "s": s, "cols": N}


def _value(a: dict, dtype: torch.dtype = torch.float32) -> torch.Tensor:
    """What stored activations [B, T, cols] stand for."""
    c = a["cols"]
    e = a["s"][..., :-(-c // BLOCK)].to(torch.int32) - 127
    return a["q"][..., :c].to(dtype) * _pow2(e).to(dtype).repeat_interleave(BLOCK, -1)[..., :c]


def _weight(a: dict, dtype: torch.dtype = torch.float32) -> torch.Tensor:
    """What a stored weight [T, K, N] stands for."""
    K, N = a["q"].shape[1], a["cols"]
    e = a["s"][..., :-(-N // BLOCK)].to(torch.int32) - 127
    s = _pow2(e).to(dtype).repeat_interleave(BLOCK, 1)[:, :K].repeat_interleave(BLOCK, 2)[..., :N]
    return a["q"][..., :N].to(dtype) * s


def _gelu(u: torch.Tensor) -> torch.Tensor:
    return 0.5 * u * torch.special.erfc(-u * math.sqrt(0.5))


def _gelu_grad(u: torch.Tensor) -> torch.Tensor:
    return 0.5 * torch.special.erfc(-u * math.sqrt(0.5)) + u * torch.exp(-0.5 * u * u) / math.sqrt(2 * math.pi)


def _per_token(x: torch.Tensor, w: torch.Tensor) -> torch.Tensor:
    """y[b, t, :] = x[b, t, :] w[t]."""
    return torch.matmul(x.transpose(0, 1), w).transpose(0, 1)


def _outer(x: torch.Tensor, y: torch.Tensor) -> torch.Tensor:
    """[t] = sum over b of x[b, t, :]^T y[b, t, :]."""
    return torch.matmul(x.permute(1, 2, 0), y.transpose(0, 1))


# ---- the cases ---------------------------------------------------------------------------------

def prepare(case: dict, seed: int) -> dict:
    g = torch.Generator(device="cuda").manual_seed(seed)
    op, B, T = case["op"], case["B"], case["T"]
    s = dict(case)
    if op == "act8":
        s["x"] = _activation(B, T, case["C"], g).to(DTYPES[case["dtype"]])
    elif op == "matmul":
        K, N = case["K"], case["N"]
        s["x"] = _act8(_activation(B, T, K, g), case["fmt"])
        s["w"] = _weight8(T, N, K, g) if case["trans"] else _weight8(T, K, N, g)
        s["bias"] = 0.1 * torch.randn((T, N), generator=g, device="cuda") if case["bias"] else None
    elif op == "wgrad":
        s["x"] = _act8(_activation(B, T, case["K"], g))
        s["dy"] = (torch.randn((B, T, case["N"]), generator=g, device="cuda") / B).to(torch.bfloat16)
    else:
        D, F = case["D"], case["F"]
        s["x"] = _activation(B, T, D, g).to(torch.bfloat16)
        s["w1"], s["w2"] = _weight8(T, D, F, g), _weight8(T, F, D, g)
        s["b1"] = 0.1 * torch.randn((T, F), generator=g, device="cuda")
        s["b2"] = 0.1 * torch.randn((T, D), generator=g, device="cuda")
        if case["train"]:
            s["dv"] = (torch.randn((B, T, D), generator=g, device="cuda") / B).to(torch.bfloat16)
        if own:                                                   # the layer that a program keeps
            from rankmixer_feature_interaction_gb300 import api
            s["ffn"] = api.Fp8PFFN(_own8(api, s["w1"]), s["b1"], _own8(api, s["w2"]), s["b2"])
    return s


def _own8(api, a: dict):
    return api.Fp8Tensor(a["q"], a["s"], a["cols"])


def _run_own(s: dict):
    from rankmixer_feature_interaction_gb300 import api
    op = s["op"]
    if op == "act8":
        return api.fp8_dequantize(api.fp8_quantize(s["x"], s["fmt"]), "bf16")
    if op == "matmul":
        return api.fp8_matmul(_own8(api, s["x"]), _own8(api, s["w"]), s["bias"], transpose_w=s["trans"])
    if op == "wgrad":
        return api.fp8_wgrad(_own8(api, s["x"]), s["dy"])
    if not s["train"]:
        return s["ffn"].forward(s["x"])
    v, kept = s["ffn"].forward_train(s["x"])
    dx, grads = s["ffn"].backward(s["dv"], kept, grad_dtype="bf16")
    return v, dx, grads["dW1"], grads["db1"], grads["dW2"], grads["db2"]


def run(s: dict):
    if own:
        return _run_own(s)
    op, b16 = s["op"], torch.bfloat16
    if op == "act8":
        return _rounded(s["x"].float(), s["fmt"]).to(b16)
    if op == "matmul":
        w = _weight(s["w"])
        y = _per_token(_value(s["x"]), w.transpose(1, 2) if s["trans"] else w)
        return (y if s["bias"] is None else y + s["bias"]).to(b16)
    if op == "wgrad":
        dy = s["dy"].float()
        return _outer(_value(s["x"]), dy), dy.sum(0)
    w1, w2 = _weight(s["w1"]), _weight(s["w2"])
    x = _rounded(s["x"].float())
    u = _per_token(x, w1) + s["b1"]
    a = _rounded(_gelu(u))
    v = (_per_token(a, w2) + s["b2"]).to(b16)
    if not s["train"]:
        return v
    u = _rounded(u)
    dv = s["dv"].float()
    du = _per_token(_rounded(dv), w2.transpose(1, 2)) * _gelu_grad(u)
    dx = _per_token(_rounded(du), w1.transpose(1, 2))
    return (v, dx.to(b16), _outer(x, du).to(b16), du.sum(0).to(b16), _outer(a, dv).to(b16), dv.sum(0).to(b16))


def work(case: dict) -> dict:
    """Each input read once, each output (and each checkpoint, which is kept) written once and read once."""
    op, rows, T = case["op"], case["B"] * case["T"], case["T"]
    e = 1 + 1 / BLOCK                                              # bytes of a value in 8 bits
    if op == "act8":
        n = rows * case["C"]
        return {"bytes": n * ((2 if case["dtype"] == "bf16" else 4) + e + e + 2), "flops": 2 * n}
    if op == "matmul":
        K, N = case["K"], case["N"]
        return {"bytes": rows * K * e + T * K * N + rows * N * 2 + (4 * T * N if case["bias"] else 0),
                "flops": 2 * rows * K * N}
    if op == "wgrad":
        K, N = case["K"], case["N"]
        return {"bytes": rows * K * e + rows * N * 2 + 4 * T * N * (K + 1), "flops": 2 * rows * K * N}
    D, F = case["D"], case["F"]
    forward = rows * D * 4 + 2 * T * D * F + 4 * T * (D + F)
    if not case["train"]:
        return {"bytes": forward, "flops": 4 * rows * D * F}
    kept = rows * (D + 2 * F) * e
    return {"bytes": forward + 2 * kept + rows * D * 4 + 2 * T * D * F + 2 * T * (2 * D * F + D + F),
            "flops": 12 * rows * D * F}


# ---- the definition in 64 bits -----------------------------------------------------------------

def _eight_bits64(x: torch.Tensor, fmt: str) -> torch.Tensor:
    """Every value of float64 rows rounded to the nearest number (ties to even) that its block's 8-bit form has:
    a whole multiple of a power of two, finer for smaller values down to the format's smallest step."""
    mantissa, largest, low = (3, 448.0, -6) if fmt == "e4m3" else (2, 57344.0, -14)
    n = x.shape[-1]
    out = torch.empty_like(x)
    for j in range(0, n, BLOCK):
        v = x[..., j:j + BLOCK]
        amax = v.abs().amax(-1, keepdim=True)
        e = torch.ceil(torch.log2(amax.clamp(min=1e-300) / largest)).clamp(min=-126)
        e = torch.where(amax <= largest * torch.exp2(e - 1), e - 1, e)       # log2's own rounding
        e = torch.where(amax > largest * torch.exp2(e), e + 1, e).clamp(min=-126)
        scaled = v / torch.exp2(e)
        step = torch.exp2((torch.frexp(scaled.abs().clamp(min=2.0 ** low))[1] - 1 - mantissa).double())
        out[..., j:j + BLOCK] = torch.round(scaled / step) * step * torch.exp2(e)
    return out


def exact(case: dict, seed: int):
    s = prepare(case, seed)
    s.pop("ffn", None)
    op, f64 = case["op"], torch.float64
    B, T = case["B"], case["T"]
    if op == "act8":
        y = torch.empty(s["x"].shape, dtype=f64, device="cuda")
        for b in range(0, B, 64):
            y[b:b + 64] = _eight_bits64(s["x"][b:b + 64].double(), case["fmt"])
        return y
    if op == "matmul":
        y = torch.empty((B, T, case["N"]), dtype=f64, device="cuda")
        for t in range(T):
            part = {"q": s["w"]["q"][t:t + 1], "s": s["w"]["s"][t:t + 1], "cols": s["w"]["cols"]}
            w = _weight(part, f64)[0]
            x = {"q": s["x"]["q"][:, t], "s": s["x"]["s"][:, t], "cols": s["x"]["cols"]}
            y[:, t] = _value(x, f64) @ (w.T if case["trans"] else w)
        return y if s["bias"] is None else y + s["bias"]
    if op == "wgrad":
        dw = torch.empty((T, case["K"], case["N"]), dtype=f64, device="cuda")
        for t in range(T):
            x = {"q": s["x"]["q"][:, t], "s": s["x"]["s"][:, t], "cols": s["x"]["cols"]}
            dw[t] = _value(x, f64).T @ s["dy"][:, t].double()
        return dw, s["dy"].double().sum(0)
    D, F = case["D"], case["F"]
    v, dx = (torch.empty((B, T, D), dtype=f64, device="cuda") for _ in range(2))
    dw1, db1 = torch.empty((T, D, F), dtype=f64, device="cuda"), torch.empty((T, F), dtype=f64, device="cuda")
    dw2, db2 = torch.empty((T, F, D), dtype=f64, device="cuda"), torch.empty((T, D), dtype=f64, device="cuda")
    for t in range(T):
        w1, w2 = (_weight({"q": a["q"][t:t + 1], "s": a["s"][t:t + 1], "cols": a["cols"]}, f64)[0]
                  for a in (s["w1"], s["w2"]))
        x = _eight_bits64(s["x"][:, t].double(), "e4m3")
        u = x @ w1 + s["b1"][t].double()
        a = _eight_bits64(u * 0.5 * torch.special.erfc(-u / math.sqrt(2.0)), "e4m3")
        v[:, t] = a @ w2 + s["b2"][t].double()
        if not case["train"]:
            continue
        u = _eight_bits64(u, "e4m3")
        slope = 0.5 * torch.special.erfc(-u / math.sqrt(2.0)) + u * torch.exp(-u * u / 2) / math.sqrt(2 * math.pi)
        dv = s["dv"][:, t].double()
        du = (_eight_bits64(dv, "e4m3") @ w2.T) * slope
        dx[:, t] = _eight_bits64(du, "e4m3") @ w1.T
        dw1[t], db1[t], dw2[t], db2[t] = x.T @ du, du.sum(0), a.T @ dv, dv.sum(0)
    return (v, dx, dw1, db1, dw2, db2) if case["train"] else v
