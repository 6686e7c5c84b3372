"""Cases, plain forms and 64-bit definitions of the operators around a feed-forward block.

What a pre-norm feed-forward block needs beside its products: root-mean-square
norm with the residual's addition, trained (with its gradients) and served (its
output in FP8 with the scales that the block-scaled product takes), that
quantisation alone for the hidden activations, dropout whose mask is never
stored, and the product of a few tokens with 4-bit weights.

A case is a dict; ``case["op"]`` names the operator:

  rms_norm  H = X + R in X's type (X alone without a residual),
            r = 1 / sqrt(mean(H^2) + eps), Y = H r gamma; returns Y, H (with a
            residual) and r.
  rms_fp8   the same with Y in FP8 (E4M3): each row's 128 columns share a scale
            S = max|Y| / 448 (1 where all are 0); returns Q, S, H.
  rms_grad  with z = H r, g = dY gamma: dX = dH + r (g - z mean(g z)) (dH, the
            gradient that comes along the residual stream, may be absent) and
            dgamma = sum dY z.
  quantize  X -> Q, S as in rms_fp8; with ``pow2`` the scales are powers of two,
            given as E8M0 bytes (2^(byte - 127)).
  dropout   Y = R + X / (1 - p) where an element is kept, R where not (R may be
            absent; the gradient is the call on dY without R).  Element e is
            kept if word e % 4 of Philox4x32-10 with counter (e / 4, offset) and
            key seed is at least floor(p 2^32).
  linear    C = ReLU(X W^T) or X W^T with W's elements s (q - z): q 4 bits, s of
            X's type and z (4 bits, 8 without zero points) for each row and
            group of columns.

Layout of 4-bit weights (N, K).  Codes: (ceil(N/16), ceil(K/64), 512) bytes.
In the 512 bytes of 16 rows and 64 columns, little-endian word 4 (4 g + t) + j
holds rows g and g + 8 (g < 8) and columns 32 (j / 2) + 8 t + 4 (j % 2) + c,
c = 0..3 (t < 4, j < 4): nibbles 0..3 are (g, c = 0), (g + 8, 0), (g, 2),
(g + 8, 2), nibbles 4..7 the same with c = 1 and 3.  Scales and zero points:
(ceil(N/16), ceil(K/group), 16), one per group and row.
"""
from __future__ import annotations

import math

import torch

own = False

DEV = "cuda:0"
DTYPES = {"fp16": torch.float16, "bf16": torch.bfloat16, "fp32": torch.float32}
EPS = 1e-6
E4M3_MAX = 448.0

LISTED = [
    # One token being generated: the norm in front of the block, adding the branch before it.
    {"name": "rms_norm_1x4096_bf16", "op": "rms_norm", "rows": 1, "dim": 4096, "type": "bf16", "wtype": "bf16",
     "residual": True},
    # A training batch.
    {"name": "rms_norm_16384x4096_fp16", "op": "rms_norm", "rows": 16384, "dim": 4096, "type": "fp16",
     "wtype": "fp16", "residual": True},
    # Ragged: a last block of 104 columns, no residual.
    {"name": "rms_fp8_1000x1000_fp32", "op": "rms_fp8", "rows": 1000, "dim": 1000, "type": "fp32", "wtype": "fp32",
     "residual": False},
    # A long prompt in front of an FP8 product.
    {"name": "rms_fp8_8192x8192_bf16", "op": "rms_fp8", "rows": 8192, "dim": 8192, "type": "bf16", "wtype": "fp32",
     "residual": True},
    # An odd width and few rows, the norm alone.
    {"name": "rms_grad_1000x1023_fp32", "op": "rms_grad", "rows": 1000, "dim": 1023, "type": "fp32",
     "wtype": "fp32", "residual": False},
    # The training batch's backward pass, with the residual stream's gradient.
    {"name": "rms_grad_16384x4096_fp16", "op": "rms_grad", "rows": 16384, "dim": 4096, "type": "fp16",
     "wtype": "fp16", "residual": True},
    # Hidden activations of a batch of 64 generated tokens.
    {"name": "quantize_64x8192_bf16", "op": "quantize", "rows": 64, "K": 8192, "type": "bf16", "pow2": False},
    # Hidden activations of a long prompt, for the product with power-of-two scales.
    {"name": "quantize_8192x8192_fp16", "op": "quantize", "rows": 8192, "K": 8192, "type": "fp16", "pow2": True},
    # A gradient of odd width.
    {"name": "dropout_1000x1001_fp32", "op": "dropout", "rows": 1000, "dim": 1001, "type": "fp32",
     "residual": False, "p": 0.5},
    # A training batch's branch added to the residual stream.
    {"name": "dropout_16384x4096_fp16", "op": "dropout", "rows": 16384, "dim": 4096, "type": "fp16",
     "residual": True, "p": 0.1},
    # One generated token.
    {"name": "linear_1x4096x4096_fp16", "op": "linear", "M": 1, "N": 4096, "K": 4096, "group": 128, "zeros": False,
     "type": "fp16", "relu": True},
    # A batch of generated tokens through a wide layer, with zero points.
    {"name": "linear_16x16384x8192_bf16", "op": "linear", "M": 16, "N": 16384, "K": 8192, "group": 64,
     "zeros": True, "type": "bf16", "relu": False},
]


def listed():
    return [dict(c) for c in LISTED]


def _log_size(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["rms_norm", "rms_fp8", "rms_grad", "quantize", "dropout", "linear"])
    if op == "linear":
        return {"op": op, "M": _log_size(rng, 1, 64), "N": _log_size(rng, 64, 16384), "K": _log_size(rng, 64, 8192),
                "group": rng.choice([32, 64, 128]), "zeros": rng.random() < 0.5, "type": rng.choice(["fp16", "bf16"]),
                "relu": rng.random() < 0.5}
    t = rng.choice(list(DTYPES))
    # No more bytes than the largest listed case has.
    most = 16384 * 4096 * 2 // DTYPES[t].itemsize
    rows = _log_size(rng, 1, 16384)
    dim = min(_log_size(rng, 64, 16384), most // rows)
    if rng.random() < 0.6:
        dim = max(64, dim // 16 * 16)   # models' widths
    if op == "quantize":
        return {"op": op, "rows": rows, "K": dim, "type": t, "pow2": rng.random() < 0.5}
    c = {"op": op, "rows": rows, "dim": dim, "type": t, "residual": rng.random() < 0.6}
    if op == "dropout":
        c["p"] = rng.choice([0.05, 0.1, 0.2, 0.5])
    else:
        c["wtype"] = rng.choice([t, "fp32"])
    return c


# ---------------------------------------------------------------- inputs


def _activations(gen, rows, dim, dtype):
    """Rows of a residual stream: unequal channels, a few of them large."""
    x = torch.randn((rows, dim), generator=gen, device=DEV)
    scale = torch.exp(0.4 * torch.randn((dim,), generator=gen, device=DEV))
    scale = scale * (1 + 15 * (torch.rand((dim,), generator=gen, device=DEV) < 0.004))
    return (x * scale).to(dtype)


def _whole(gen, bits):
    """A number of so many bits."""
    return int(torch.randint(0, 2 ** bits, (1,), generator=gen, device=DEV).item())


def prepare(case, seed):
    gen = torch.Generator(device=DEV)
    gen.manual_seed(seed)
    op = case["op"]
    st = {"case": dict(case)}
    dtype = DTYPES[case["type"]]
    if op == "quantize":
        st["X"] = _activations(gen, case["rows"], case["K"], dtype)
        return st
    if op == "linear":
        M, N, K, G = case["M"], case["N"], case["K"], case["group"]
        groups = -(-K // G)
        st["X"] = _activations(gen, M, K, dtype)
        q = torch.randint(0, 16, (N, K), generator=gen, device=DEV, dtype=torch.uint8)
        # Elements of size 1 / sqrt(K), the groups' ranges unequal.
        s = torch.exp(0.3 * torch.randn((N, groups), generator=gen, device=DEV)) / (4.6 * math.sqrt(K))
        z = torch.randint(5, 11, (N, groups), generator=gen, device=DEV, dtype=torch.uint8)
        st["Q"], st["S"] = _tile_codes(q), _tile_groups(s.to(dtype))
        st["Z"] = _tile_groups(z) if case["zeros"] else None
        return st
    rows, dim = case["rows"], case["dim"]
    st["X"] = _activations(gen, rows, dim, dtype)
    st["R"] = _activations(gen, rows, dim, dtype) if case["residual"] else None
    if op == "dropout":
        st["seed"], st["offset"] = _whole(gen, 62), _whole(gen, 40)
        return st
    st["gamma"] = (1 + 0.1 * torch.randn((dim,), generator=gen, device=DEV)).to(DTYPES[case["wtype"]])
    if op == "rms_grad":
        # X is the stream that the forward pass kept, with the statistic; R the gradient along it.
        st["rstd"] = _rstd_plain(st["X"])
        st["dY"] = torch.randn((rows, dim), generator=gen, device=DEV).to(dtype)
    return st


# ---------------------------------------------------------------- 4-bit weights' layout


def _pad(x, rows, cols):
    return torch.nn.functional.pad(x, (0, cols - x.shape[1], 0, rows - x.shape[0]))


def _tile_codes(q):
    """Codes (N, K), a byte each, in the packed layout; what fills up the tiles is zero."""
    N, K = q.shape
    nt, kt = -(-N // 16), -(-K // 64)
    # row = 8 hi + g, column = 32 h + 8 t + 4 i + 2 c1 + c0
    q = _pad(q, nt * 16, kt * 64).reshape(nt, 2, 8, kt, 2, 4, 2, 2, 2)
    # nibble = 4 c0 + 2 c1 + hi of word 4 (4 g + t) + 2 h + i
    q = q.permute(0, 3, 2, 5, 4, 6, 8, 7, 1).reshape(nt, kt, 512, 2)
    return (q[..., 0] | (q[..., 1] << 4)).contiguous()


def _untile_codes(Q, N, K):
    nt, kt = Q.shape[:2]
    q = torch.stack([Q & 15, Q >> 4], dim=-1).reshape(nt, kt, 8, 4, 2, 2, 2, 2, 2)
    return q.permute(0, 8, 2, 1, 4, 3, 5, 7, 6).reshape(nt * 16, kt * 64)[:N, :K]


def _tile_groups(s):
    """One value per row and group, (N, groups), as (ceil(N/16), groups, 16)."""
    nt = -(-s.shape[0] // 16)
    return _pad(s, nt * 16, s.shape[1]).reshape(nt, 16, -1).transpose(1, 2).contiguous()


def _untile_groups(S, N):
    return S.transpose(1, 2).reshape(S.shape[0] * 16, -1)[:N]


# ---------------------------------------------------------------- plain forms


def _rstd_plain(h):
    h = h.float()
    return 1.0 / torch.sqrt((h * h).mean(dim=1) + EPS)


def _fp8_plain(y, pow2=False):
    """E4M3 elements and scales of fp32 rows, blocks of 128 columns."""
    rows, K = y.shape
    KB = -(-K // 128)
    b = torch.nn.functional.pad(y, (0, KB * 128 - K)).reshape(rows, KB, 128)
    a = b.abs().amax(dim=2)
    if pow2:
        # The least e with a <= 448 2^e, from a = m 2^x with m in [0.5, 1) and 448 = 0.875 2^9.
        m, x = torch.frexp(a)
        e = torch.where(a > 0, x - 9 + (m > 0.875).int(), torch.zeros_like(x)).clamp(-127, 127)
        h = torch.div(-e, 2, rounding_mode="floor")
        q = b * _pow2(h)[:, :, None] * _pow2(-e - h)[:, :, None]
        s = (e + 127).to(torch.uint8)
    else:
        # 448 b / a with one rounding where 7/8 b is exact (16-bit rows), so that ties stay ties.
        q = (0.875 * b) / torch.where(a > 0, a, torch.ones_like(a))[:, :, None] * 512.0
        s = torch.where(a > 0, a / E4M3_MAX, torch.ones_like(a))
    q = q.clamp(-E4M3_MAX, E4M3_MAX).reshape(rows, KB * 128)[:, :K]
    return q.to(torch.float8_e4m3fn), s


def _pow2(e):
    """2^e in fp32, exactly, for whole numbers -126 <= e <= 127."""
    return ((e.to(torch.int32) + 127) << 23).view(torch.float32)


def _philox_plain(n, seed, offset):
    """The first n 32-bit words, as int64: Philox4x32-10 of counters (0, offset), (1, offset), ..."""
    m32 = 0xFFFFFFFF
    i = torch.arange(-(-n // 4), device=DEV, dtype=torch.int64)
    c0, c1 = i & m32, i >> 32
    c2, c3 = torch.full_like(i, offset & m32), torch.full_like(i, offset >> 32)
    k0, k1 = seed & m32, seed >> 32
    for _ in range(10):
        # Products of 32-bit numbers: int64 wraps, its bits are those of the whole product.
        p0, p1 = c0 * 0xD2511F53, c2 * 0xCD9E8D57
        c0, c1, c2, c3 = ((p1 >> 32) & m32) ^ c1 ^ k0, p1 & m32, ((p0 >> 32) & m32) ^ c3 ^ k1, p0 & m32
        k0, k1 = (k0 + 0x9E3779B9) & m32, (k1 + 0xBB67AE85) & m32
    return torch.stack([c0, c1, c2, c3], dim=1).reshape(-1)[:n]


def run(state):
    return _run_own(state) if own else _run_plain(state)


def _run_plain(state):
    c = state["case"]
    op = c["op"]
    X, dtype = state["X"], state["X"].dtype
    if op == "quantize":
        return _fp8_plain(X.float(), c["pow2"])
    if op == "linear":
        N, K, G = c["N"], c["K"], c["group"]
        s = _untile_groups(state["S"], N).float().repeat_interleave(G, dim=1)[:, :K]
        z = 8.0 if state["Z"] is None else _untile_groups(state["Z"], N).float().repeat_interleave(G, dim=1)[:, :K]
        y = X.float() @ ((_untile_codes(state["Q"], N, K).float() - z) * s).t()
        return (torch.clamp(y, min=0) if c["relu"] else y).to(dtype)
    R = state["R"]
    if op == "dropout":
        keep = (_philox_plain(X.numel(), state["seed"], state["offset"]) >= int(c["p"] * 2 ** 32)).reshape(X.shape)
        y = torch.where(keep, X.float() * (1.0 / (1.0 - c["p"])), torch.zeros((), device=DEV))
        return (y if R is None else R.float() + y).to(dtype)
    gamma = state["gamma"].float()
    if op == "rms_grad":
        z = X.float() * state["rstd"][:, None]
        dy = state["dY"].float()
        g = dy * gamma
        dx = state["rstd"][:, None] * (g - z * (g * z).mean(dim=1, keepdim=True))
        if R is not None:
            dx = R.float() + dx
        # Sums over all rows, with terms of both signs: in 64 bits.
        return dx.to(dtype), (dy * z).sum(dim=0, dtype=torch.float64).to(state["gamma"].dtype)
    h = X if R is None else (X.float() + R.float()).to(dtype)
    r = _rstd_plain(h)
    y = h.float() * r[:, None] * gamma
    if op == "rms_fp8":
        q, s = _fp8_plain(y)
        return q, s, None if R is None else h
    return y.to(dtype), None if R is None else h, r


def _run_own(state):
    from dense_fp16_gemm_05_gb300 import gemm_f16 as g

    c = state["case"]
    op = c["op"]
    X = state["X"]
    if op == "quantize":
        return g.fp8_quantize(X, pow2=c["pow2"])
    if op == "linear":
        return g.linear_w4(X, state["Q"], state["S"], state["Z"], N=c["N"], group=c["group"], relu=c["relu"])
    R = state["R"]
    if op == "dropout":
        return g.dropout(X, c["p"], state["seed"], state["offset"], residual=R)
    if op == "rms_grad":
        return g.rms_norm_bwd(state["dY"], X, state["rstd"], state["gamma"], dH=R)
    if op == "rms_fp8":
        q, s, h = g.rms_norm_fp8(X, state["gamma"], residual=R, eps=EPS)
        return q, s, None if R is None else h
    y, h, r = g.rms_norm_fwd(X, state["gamma"], residual=R, eps=EPS)
    return y, None if R is None else h, r


# ---------------------------------------------------------------- work


def work(case):
    op, el = case["op"], DTYPES[case["type"]].itemsize
    if op == "quantize":
        rows, K = case["rows"], case["K"]
        return {"bytes": rows * K * (el + 1) + rows * -(-K // 128) * (1 if case["pow2"] else 4), "flops": 3 * rows * K}
    if op == "linear":
        M, N, K = case["M"], case["N"], case["K"]
        groups = -(-K // case["group"])
        return {"bytes": N * K / 2 + N * groups * (el + bool(case["zeros"])) + 2 * M * (N + K), "flops": 2 * M * N * K}
    rows, dim = case["rows"], case["dim"]
    n, res = rows * dim, bool(case["residual"])
    if op == "dropout":
        return {"bytes": n * el * (2 + res), "flops": 3 * n}
    wel = DTYPES[case["wtype"]].itemsize
    if op == "rms_grad":
        return {"bytes": n * el * (3 + res) + 2 * dim * wel + 4 * rows, "flops": 10 * n}
    out = 1 if op == "rms_fp8" else el
    stat = rows * -(-dim // 128) * 4 if op == "rms_fp8" else rows * 4
    return {"bytes": n * (el * (1 + 2 * res) + out) + dim * wel + stat, "flops": 6 * n}


# ---------------------------------------------------------------- the definitions in 64 bits


def _e4m3_nearest(v):
    """The nearest E4M3 number of every element of |v| <= 448: steps of 2^(x - 3) from 2^x on, 2^-9 below 2^-6."""
    x = torch.floor(torch.log2(v.abs().clamp(min=2.0 ** -6)))
    step = torch.exp2(x.clamp(min=-6.0) - 3)
    # rint: to the even multiple at a tie.
    return torch.round(v / step) * step


def _fp8_exact(y, pow2=False):
    rows, K = y.shape
    scales, values = [], []
    for b in range(0, K, 128):
        blk = y[:, b:b + 128]
        a = blk.abs().amax(dim=1)
        one = torch.ones_like(a)
        s = torch.where(a > 0, a / 448, one)
        if pow2:
            e = torch.ceil(torch.log2(s))
            e = torch.where(torch.exp2(e - 1) * 448 >= a, e - 1, e)   # the logarithm's error
            e = torch.where(torch.exp2(e) * 448 < a, e + 1, e)
            e = torch.where(a > 0, e, torch.zeros_like(e)).clamp(-127, 127)
            s = torch.exp2(e)
            scales.append((e + 127).to(torch.uint8))
            v = blk / s[:, None]
        else:
            scales.append(s)
            v = blk * 448 / torch.where(a > 0, a, one)[:, None]   # blk / s without s's rounding, which breaks ties
        values.append(_e4m3_nearest(v.clamp(-448, 448)))
    return torch.cat(values, dim=1), torch.stack(scales, dim=1)


def _philox_words(n, seed, offset):
    """The same words by 16-bit limbs, without a product of more than 33 bits."""
    def mulhilo(a, b):
        al, ah, bl, bh = a & 0xFFFF, a >> 16, b & 0xFFFF, b >> 16
        mid = ah * bl + ((al * bl) >> 16)
        mid2 = al * bh + (mid & 0xFFFF)
        return ah * bh + (mid >> 16) + (mid2 >> 16), ((mid2 & 0xFFFF) << 16) | ((al * bl) & 0xFFFF)

    i = torch.arange((n + 3) // 4, device=DEV, dtype=torch.int64)
    x = [i % 2 ** 32, i // 2 ** 32, i * 0 + offset % 2 ** 32, i * 0 + offset // 2 ** 32]
    for rnd in range(10):
        ka = (seed % 2 ** 32 + rnd * 0x9E3779B9) % 2 ** 32
        kb = (seed // 2 ** 32 + rnd * 0xBB67AE85) % 2 ** 32
        h0, l0 = mulhilo(x[0], 0xD2511F53)
        h1, l1 = mulhilo(x[2], 0xCD9E8D57)
        x = [h1 ^ x[1] ^ ka, l1, h0 ^ x[3] ^ kb, l0]
    out = torch.empty((len(i), 4), dtype=torch.int64, device=DEV)
    for w in range(4):
        out[:, w] = x[w]
    return out.flatten()[:n]


def exact(case, seed):
    st = prepare(case, seed)
    op, X = case["op"], st["X"]
    x = X.double()
    if op == "quantize":
        return _fp8_exact(x, case["pow2"])
    if op == "linear":
        N, K, G = case["N"], case["K"], case["group"]
        n = torch.arange(N, device=DEV)[:, None]
        out = torch.zeros((case["M"], N), dtype=torch.float64, device=DEV)
        for k0 in range(0, K, G):
            k = torch.arange(k0, min(k0 + G, K), device=DEV)[None, :]
            c, kk = k % 4, k % 64
            word = 4 * (4 * (n % 8) + kk % 32 // 8) + 2 * (kk // 32) + kk % 8 // 4
            nibble = 4 * (c % 2) + 2 * (c // 2) + n % 16 // 8
            q = (st["Q"][n // 16, k // 64, 4 * word + nibble // 2].long() >> (4 * (nibble % 2))) & 15
            z = 8 if st["Z"] is None else st["Z"][n // 16, k0 // G, n % 16].double()
            w = (q.double() - z) * st["S"][n // 16, k0 // G, n % 16].double()
            out += x[:, k0:k0 + G] @ w.t()
        return out * (out > 0) if case["relu"] else out
    R = st["R"]
    if op == "dropout":
        keep = (_philox_words(X.numel(), st["seed"], st["offset"]) >= math.floor(case["p"] * 2 ** 32)).reshape(X.shape)
        y = x * keep / (1 - case["p"])
        return y if R is None else y + R.double()
    gamma = st["gamma"].double()
    n = case["dim"]
    if op == "rms_grad":
        r, dy = st["rstd"].double()[:, None], st["dY"].double()
        gz = dy * gamma * x
        dx = dy * gamma * r - x * r ** 3 * (gz.sum(1, keepdim=True) / n)
        return dx if R is None else dx + R.double(), (dy * x * r).sum(0)
    # The stream is kept in its type, and its norm is taken of that.
    h = X if R is None else (x + R.double()).to(X.dtype)
    hd = h.double()
    r = (hd.square().sum(1) / n + EPS).rsqrt()
    y = hd * r[:, None] * gamma
    kept = None if R is None else hd
    if op == "rms_fp8":
        q, s = _fp8_exact(y)
        return q, s, kept
    return y, kept, r
