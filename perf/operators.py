"""Cases, plain forms and 64-bit definitions of the feed-forward operators.

The operators are those of a pre-norm feed-forward layer, served in 4 bits and
trained in 16: microscaled 4-bit floating point (MXFP4: E2M1 elements, one
power-of-two E8M0 scale per 32 elements), its quantisation and its product
with the fused ReLU, and layer norm with its gradients.

A case is a dict; ``case["op"]`` names the operator:

  quantize  X (rows, K) -> what its MXFP4 form stands for (rows, K).  With
            ``trans`` X is stored (K, rows) and its columns are quantised (a
            weight stored in-features x out-features).
  product   C = R(A @ W^T) from MXFP4 operands, C fp16.
  linear    the same with A quantised from 16-bit activations in the call.
  norm      layer norm: Y, mean, 1/sqrt(variance + eps).
  norm_grad its gradients: dX, dgamma, dbeta.

Layout of a quantised (rows, K) matrix.  Codes: (rows, 16 ceil(K/32)) bytes,
element 2i in the low half of byte i.  Scales: (ceil(rows/128),
ceil(K/128), 512) bytes, the E8M0 byte of row r and block b (32 elements) at
tile [r // 128, b // 4], byte (r % 32) * 16 + (r % 128 // 32) * 4 + b % 4.
"""
from __future__ import annotations

import math

import torch

own = False

DEV = "cuda:0"
DTYPES = {"fp16": torch.float16, "bf16": torch.bfloat16, "fp32": torch.float32}
EPS = 1e-5

LISTED = [
    # One row of activations of a token being generated, kept with its codes.
    {"name": "quantize_1x4096_bf16", "op": "quantize", "rows": 1, "K": 4096, "type": "bf16", "trans": False},
    # Ragged in both sizes: the last block of a row is partly filled.
    {"name": "quantize_1000x1000_fp32", "op": "quantize", "rows": 1000, "K": 1000, "type": "fp32", "trans": False},
    # A long batch's activations.
    {"name": "quantize_8192x8192_fp16", "op": "quantize", "rows": 8192, "K": 8192, "type": "fp16", "trans": False},
    # A weight stored (in, out), quantised along in.
    {"name": "quantize_trans_4096x4096_fp16", "op": "quantize", "rows": 4096, "K": 4096, "type": "fp16",
     "trans": True},
    # One generated token: bound by reading the weight.
    {"name": "linear_1x4096x4096_fp16", "op": "linear", "M": 1, "N": 4096, "K": 4096, "relu": True, "type": "fp16"},
    # A batch of 64 generated tokens.
    {"name": "linear_64x8192x4096_bf16", "op": "linear", "M": 64, "N": 8192, "K": 4096, "relu": True, "type": "bf16"},
    # Ragged in every size.
    {"name": "product_1000x1000x1000", "op": "product", "M": 1000, "N": 1000, "K": 1000, "relu": True},
    # The largest: a long prompt through a wide layer.
    {"name": "product_8192x8192x8192", "op": "product", "M": 8192, "N": 8192, "K": 8192, "relu": True},
    # A few rows, fp32 weights of the norm beside 16-bit activations.
    {"name": "norm_64x4096_bf16_fp32", "op": "norm", "rows": 64, "dim": 4096, "type": "bf16", "wtype": "fp32"},
    # A training batch.
    {"name": "norm_16384x4096_fp16", "op": "norm", "rows": 16384, "dim": 4096, "type": "fp16", "wtype": "fp16"},
    # An odd width and few rows.
    {"name": "norm_grad_1000x1023_fp32", "op": "norm_grad", "rows": 1000, "dim": 1023, "type": "fp32",
     "wtype": "fp32"},
    # The training batch's backward pass.
    {"name": "norm_grad_16384x4096_fp16", "op": "norm_grad", "rows": 16384, "dim": 4096, "type": "fp16",
     "wtype": "fp16"},
]


def listed():
    return [dict(c) for c in LISTED]


def _log_size(rng, lo, hi, step=1):
    v = int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))
    return max(lo, min(hi, (v + step - 1) // step * step))


def draw(rng):
    op = rng.choice(["quantize", "product", "linear", "norm", "norm_grad"])
    if op == "quantize":
        # Beyond the largest listed matrix no draw.
        rows = _log_size(rng, 1, 16384)
        K = min(_log_size(rng, 32, 16384), 8192 * 8192 // rows)
        return {"op": op, "rows": rows, "K": K, "type": rng.choice(list(DTYPES)), "trans": rng.random() < 0.3}
    if op in ("product", "linear"):
        M = _log_size(rng, 1, 8192)
        N = _log_size(rng, 64, 8192, 8)
        K = _log_size(rng, 64, 8192)
        c = {"op": op, "M": M, "N": N, "K": K, "relu": rng.random() < 0.7}
        if op == "linear":
            c["type"] = rng.choice(["fp16", "bf16"])
        return c
    rows = _log_size(rng, 1, 16384)
    dim = min(_log_size(rng, 64, 16384), 16384 * 4096 // rows)
    t = rng.choice(list(DTYPES))
    return {"op": op, "rows": rows, "dim": dim, "type": t, "wtype": rng.choice([t, "fp32"])}


# ---------------------------------------------------------------- MXFP4 in elementary operations


def _pow2(e):
    """2^e in fp32, exactly, for whole numbers -126 <= e <= 127."""
    return ((e.to(torch.int32) + 127) << 23).view(torch.float32)


def _encode_plain(X, trans):
    """Codes' magnitudes with sign (as values of E2M1) and block exponents of X in fp32.

    Block scale 2^e with e = floor(log2(max |x|)) - 2 (E2M1's largest exponent
    is 2), kept within E8M0's range; elements rounded to the nearest E2M1
    value, ties to even, beyond 6 to 6.  K is filled up with zeros to whole
    blocks.
    """
    x = X.float()
    if trans:
        x = x.t()
    rows, K = x.shape
    KB = -(-K // 32)
    x = torch.nn.functional.pad(x, (0, KB * 32 - K)).reshape(rows, KB, 32)
    e = torch.frexp(x.abs().amax(dim=2))[1] - 3          # frexp's mantissa lies in [0.5, 1)
    e = torch.where((x == 0).all(dim=2), torch.full_like(e, -127), e).clamp(-127, 127)
    # 2^-e in two factors: each is a normal number.
    h = torch.div(-e, 2, rounding_mode="floor")
    v = x * _pow2(h)[:, :, None] * _pow2(-e - h)[:, :, None]
    a = v.abs()
    mag = (0.5 * ((a > 0.25).float() + (a >= 0.75) + (a > 1.25) + (a >= 1.75))
           + (a > 2.5) + (a >= 3.5) + 2.0 * (a > 5.0))
    return torch.where(v < 0, -mag, mag), e


def _values_plain(X, trans):
    """fp32 values that the MXFP4 form of X stands for, (rows, K)."""
    val, e = _encode_plain(X, trans)
    K = X.shape[0] if trans else X.shape[1]
    # 2^e in two factors: 2^-127 is below fp32's normal range.
    h = torch.div(e, 2, rounding_mode="floor")
    val = val * _pow2(h)[:, :, None] * _pow2(e - h)[:, :, None]
    return val.reshape(val.shape[0], -1)[:, :K]


def _pack(val, e):
    """Codes and scale tiles from E2M1 values (rows, KB, 32) and exponents (rows, KB)."""
    rows, KB = e.shape
    a = val.abs()
    code = ((2 * a).to(torch.uint8) * (a <= 2) + (a == 3) * 5 + (a == 4) * 6 + (a == 6) * 7).to(torch.uint8)
    code = code + 8 * (val < 0).to(torch.uint8)
    code = code.reshape(rows, KB * 16, 2)
    q = code[:, :, 0] + 16 * code[:, :, 1]
    RB, KA = -(-rows // 128), -(-KB // 4)
    s = torch.zeros((RB * 128, KA * 4), dtype=torch.uint8, device=e.device)
    s[:rows, :KB] = (e + 127).to(torch.uint8)
    s = s.reshape(RB, 4, 32, KA, 4).permute(0, 3, 2, 1, 4).contiguous().reshape(RB, KA, 512)
    return q.contiguous(), s


def _unpack(q, s, rows, K):
    """fp32 values of codes and scale tiles, (rows, K)."""
    RB, KA = s.shape[0], s.shape[1]
    KB = -(-K // 32)
    e = s.reshape(RB, KA, 32, 4, 4).permute(0, 3, 2, 1, 4).reshape(RB * 128, KA * 4)[:rows, :KB].to(torch.int32) - 127
    table = torch.tensor([0, 0.5, 1, 1.5, 2, 3, 4, 6], device=q.device)
    table = torch.cat([table, -table])
    code = torch.stack([q & 15, q >> 4], dim=2).reshape(rows, KB, 32)
    h = torch.div(e, 2, rounding_mode="floor")
    v = table[code.int()] * _pow2(h)[:, :, None] * _pow2(e - h)[:, :, None]
    return v.reshape(rows, KB * 32)[:, :K]


# ---------------------------------------------------------------- inputs


def _activations(gen, rows, dim, dtype):
    """Rows of a residual stream: unequal channels, a few of them large, and a mean."""
    x = torch.randn((rows, dim), generator=gen, device=DEV)
    scale = torch.exp(0.4 * torch.randn((dim,), generator=gen, device=DEV))
    scale = scale * (1 + 15 * (torch.rand((dim,), generator=gen, device=DEV) < 0.004))
    shift = 0.2 * torch.randn((dim,), generator=gen, device=DEV)
    return (x * scale + shift).to(dtype)


def prepare(case, seed):
    gen = torch.Generator(device=DEV)
    gen.manual_seed(seed)
    op = case["op"]
    st = {"case": dict(case)}
    if op == "quantize":
        shape = (case["K"], case["rows"]) if case["trans"] else (case["rows"], case["K"])
        st["X"] = _activations(gen, *shape, DTYPES[case["type"]])
    elif op in ("product", "linear"):
        M, N, K = case["M"], case["N"], case["K"]
        X = _activations(gen, M, K, DTYPES[case.get("type", "fp16")])
        W = torch.randn((N, K), generator=gen, device=DEV) / math.sqrt(K)
        st["W"], st["SW"] = _pack(*_encode_plain(W, False))
        if op == "linear":
            st["X"] = X
        else:
            st["A"], st["SA"] = _pack(*_encode_plain(X, False))
    else:
        rows, dim, wt = case["rows"], case["dim"], DTYPES[case["wtype"]]
        st["X"] = _activations(gen, rows, dim, DTYPES[case["type"]])
        st["gamma"] = (1 + 0.1 * torch.randn((dim,), generator=gen, device=DEV)).to(wt)
        st["beta"] = (0.1 * torch.randn((dim,), generator=gen, device=DEV)).to(wt)
        if op == "norm_grad":
            st["dY"] = torch.randn((rows, dim), generator=gen, device=DEV).to(DTYPES[case["type"]])
            # The statistics that the forward pass kept.
            _, st["mean"], st["rstd"] = _norm_plain(st["X"], st["gamma"], st["beta"])
    return st


# ---------------------------------------------------------------- plain forms


def _norm_plain(X, gamma, beta):
    x = X.float()
    mean = x.mean(dim=1)
    xc = x - mean[:, None]
    rstd = 1.0 / torch.sqrt((xc * xc).mean(dim=1) + EPS)
    y = xc * rstd[:, None] * gamma.float() + beta.float()
    return y.to(X.dtype), mean, rstd


def _norm_grad_plain(dY, X, gamma, mean, rstd):
    dy = dY.float()
    xhat = (X.float() - mean[:, None]) * rstd[:, None]
    g = dy * gamma.float()
    c1 = g.mean(dim=1)
    c2 = (g * xhat).mean(dim=1)
    dx = rstd[:, None] * (g - c1[:, None] - xhat * c2[:, None])
    # Sums over all rows, with terms of both signs: in 64 bits.
    dgamma = (dy * xhat).sum(dim=0, dtype=torch.float64)
    dbeta = dy.sum(dim=0, dtype=torch.float64)
    return dx.to(X.dtype), dgamma.to(gamma.dtype), dbeta.to(gamma.dtype)


def run(state):
    return _run_own(state) if own else _run_plain(state)


def _run_plain(state):
    c = state["case"]
    op = c["op"]
    if op == "quantize":
        return _values_plain(state["X"], c["trans"]).to(state["X"].dtype)
    if op in ("product", "linear"):
        M, N, K = c["M"], c["N"], c["K"]
        a = _values_plain(state["X"], False) if op == "linear" else _unpack(state["A"], state["SA"], M, K)
        y = a @ _unpack(state["W"], state["SW"], N, K).t()
        if c["relu"]:
            y = torch.clamp(y, min=0)
        return y.half()
    if op == "norm":
        return _norm_plain(state["X"], state["gamma"], state["beta"])
    return _norm_grad_plain(state["dY"], state["X"], state["gamma"], state["mean"], state["rstd"])


def _run_own(state):
    from dense_fp16_gemm_05_gb300 import gemm_f16 as g

    c = state["case"]
    op = c["op"]
    if op == "quantize":
        return g.mxfp4_quantize(state["X"], transpose=c["trans"], values=True)[2]
    if op == "product":
        return g.gemm_mxfp4(state["A"], state["SA"], state["W"], state["SW"], K=c["K"], relu=c["relu"])
    if op == "linear":
        A, SA = g.mxfp4_quantize(state["X"])
        return g.gemm_mxfp4(A, SA, state["W"], state["SW"], K=c["K"], relu=c["relu"])
    if op == "norm":
        return g.layer_norm_fwd(state["X"], state["gamma"], state["beta"], eps=EPS)
    return g.layer_norm_bwd(state["dY"], state["X"], state["mean"], state["rstd"], state["gamma"])


# ---------------------------------------------------------------- work


def work(case):
    op = case["op"]
    if op == "quantize":
        n, el = case["rows"] * case["K"], DTYPES[case["type"]].itemsize
        # X in; codes, scales and the values they stand for out.
        packed = case["rows"] * -(-case["K"] // 32) * 17
        return {"bytes": 2 * n * el + packed, "flops": 4 * n}
    if op in ("product", "linear"):
        M, N, K = case["M"], case["N"], case["K"]
        per_row = -(-K // 32) * 17
        a = M * K * 2 if op == "linear" else M * per_row
        return {"bytes": a + N * per_row + 2 * M * N, "flops": 2 * M * N * K}
    rows, dim = case["rows"], case["dim"]
    el, wel = DTYPES[case["type"]].itemsize, DTYPES[case["wtype"]].itemsize
    if op == "norm":
        return {"bytes": 2 * rows * dim * el + 2 * dim * wel + 8 * rows, "flops": 8 * rows * dim}
    return {"bytes": 3 * rows * dim * el + 3 * dim * wel + 8 * rows, "flops": 15 * rows * dim}


# ---------------------------------------------------------------- the definitions in 64 bits


def _two_to(k):
    """2^k in 64 bits, exactly, for whole numbers of any float type."""
    return ((k.to(torch.int64) + 1023) << 52).view(torch.float64)


def _exact_values(X, trans):
    """The nearest representable value of every element, by search over E2M1's eight magnitudes."""
    x = (X.t() if trans else X).double()
    rows, K = x.shape
    out = torch.empty((rows, K), dtype=torch.float64, device=x.device)
    grid = torch.tensor([0, 0.5, 1, 1.5, 2, 3, 4, 6], dtype=torch.float64, device=x.device)
    mid = (grid[1:] + grid[:-1]) / 2
    for b in range(0, K, 32):
        blk = x[:, b:b + 32]
        m = blk.abs().max(dim=1, keepdim=True).values
        # floor(log2(m)) of a number with at most 24 significant bits: the log's
        # error is put right by comparing with the power itself.
        k = torch.floor(torch.log2(m.clamp(min=1e-45)))
        k = torch.where(_two_to(k) > m, k - 1, k)
        k = torch.where(_two_to(k + 1) <= m, k + 1, k)
        s = _two_to((k - 2).clamp(-127, 127))
        v = blk.abs() / s
        lo = torch.bucketize(v.contiguous(), mid)                      # v == mid[i] gives i, the lower neighbour
        tie = (v == mid[lo.clamp(max=6)]) & (lo < 7) & (lo % 2 == 1)   # an odd code is not even: go up
        out[:, b:b + 32] = torch.sign(blk) * grid[lo + tie.long()] * s
    return out


def _exact_decode(q, s, rows, K):
    """Elements and scales of the packed form by their bit fields."""
    out = torch.empty((rows, K), dtype=torch.float64, device=q.device)
    r = torch.arange(rows, device=q.device)
    for b in range(-(-K // 32)):
        byte = s[r // 128, b // 4, (r % 32) * 16 + (r % 128) // 32 * 4 + b % 4]
        k = torch.arange(b * 32, min(b * 32 + 32, K), device=q.device)
        nib = (q[:, k // 2] >> (4 * (k % 2)).to(torch.uint8)[None, :]) & 15
        ex, man = ((nib >> 1) & 3).double(), (nib & 1).double()
        mag = torch.where(ex > 0, _two_to(ex - 1) * (1 + man / 2), man / 2)
        out[:, k] = torch.where(nib >= 8, -mag, mag) * _two_to(byte.long() - 127)[:, None]
    return out


def exact(case, seed):
    st = prepare(case, seed)
    op = case["op"]
    if op == "quantize":
        return _exact_values(st["X"], case["trans"])
    if op in ("product", "linear"):
        M, N, K = case["M"], case["N"], case["K"]
        a = _exact_values(st["X"], False) if op == "linear" else _exact_decode(st["A"], st["SA"], M, K)
        y = torch.matmul(a, _exact_decode(st["W"], st["SW"], N, K).t())
        return y * (y > 0) if case["relu"] else y
    x, w = st["X"].double(), st["gamma"].double()
    n = x.shape[1]
    if op == "norm":
        mu = x.sum(1) / n
        var = (x - mu[:, None]).square().sum(1) / n
        r = (var + EPS).rsqrt()
        return (x - mu[:, None]) * r[:, None] * w + st["beta"].double(), mu, r
    mu, r, dy = st["mean"].double(), st["rstd"].double(), st["dY"].double()
    z = (x - mu[:, None]) * r[:, None]
    gz = dy * w
    dx = (gz - (gz.sum(1, keepdim=True) + z * (gz * z).sum(1, keepdim=True)) / n) * r[:, None]
    return dx, (dy * z).sum(0), dy.sum(0)
