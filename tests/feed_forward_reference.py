"""Plain restatements, in 64 bits or whole numbers, of what the operators around a
feed-forward block compute: E4M3 block quantisation, the dropout mask, 4-bit weights.

Written from the definitions in include/gemm_f16.h, without the library.
"""
from __future__ import annotations

import torch

M32 = 0xFFFFFFFF


def philox_words(counter: list[int], key: list[int], rounds: int = 10) -> list[int]:
    """Philox4x32 of one counter (four 32-bit words) and key (two), on Python's whole numbers."""
    c, k = list(counter), list(key)
    for _ in range(rounds):
        p0, p1 = c[0] * 0xD2511F53, c[2] * 0xCD9E8D57
        c = [(p1 >> 32) ^ c[1] ^ k[0], p1 & M32, (p0 >> 32) ^ c[3] ^ k[1], p0 & M32]
        k = [(k[0] + 0x9E3779B9) & M32, (k[1] + 0xBB67AE85) & M32]
    return c


def kept(first: int, n: int, p: float, seed: int, offset: int) -> torch.Tensor:
    """Which of the elements first .. first + n - 1 dropout keeps."""
    out = []
    for e in range(first, first + n):
        if e == first or e % 4 == 0:
            i = e // 4
            words = philox_words([i & M32, i >> 32, offset & M32, offset >> 32], [seed & M32, seed >> 32])
        out.append(words[e % 4] >= int(p * 2 ** 32))
    return torch.tensor(out)


def e4m3_half_step(v: torch.Tensor) -> torch.Tensor:
    """Half the distance between E4M3 numbers at |v|: three bits behind the point, 2^-9 below 2^-6."""
    e = torch.floor(torch.log2(v.abs().clamp(min=2.0 ** -6)))
    return torch.exp2(e - 4)


def blocks(x: torch.Tensor, block_rows: int) -> torch.Tensor:
    """x (rows, K) in 64 bits as (row blocks, block_rows, column blocks, 128), filled up with zeros."""
    rows, K = x.shape
    RB, KB = -(-rows // block_rows), -(-K // 128)
    full = torch.zeros((RB * block_rows, KB * 128), dtype=torch.float64, device=x.device)
    full[:rows, :K] = x
    return full.reshape(RB, block_rows, KB, 128)


def spread(s: torch.Tensor, block_rows: int, rows: int, K: int) -> torch.Tensor:
    """A value per block as one per element."""
    return s.repeat_interleave(block_rows, 0).repeat_interleave(128, 1)[:rows, :K]


def unpack_w4(Q: torch.Tensor, N: int, K: int) -> torch.Tensor:
    """Codes (N, K) of packed 4-bit weights, by the header's words and nibbles."""
    n = torch.arange(N, device=Q.device)[:, None]
    k = torch.arange(K, device=Q.device)[None, :]
    r, kk = n % 16, k % 64
    g, b = r % 8, r // 8
    t, h, i, c = kk % 32 // 8, kk // 32, kk % 8 // 4, kk % 4
    word = 4 * (4 * g + t) + 2 * h + i
    nibble = 4 * (c % 2) + 2 * (c // 2) + b
    byte = Q[n // 16, k // 64, 4 * word + nibble // 2].long()
    return byte >> (4 * (nibble % 2)) & 15


def per_column(S: torch.Tensor, N: int, K: int, group: int) -> torch.Tensor:
    """Scales or zero points (strips, groups, 16) as (N, K) in 64 bits."""
    s = S.transpose(1, 2).reshape(-1, S.shape[1])[:N].double()
    return s.repeat_interleave(group, 1)[:, :K]


def weight_w4(Q, S, Z, N: int, K: int, group: int) -> torch.Tensor:
    """The weight (N, K) that a packed form stands for, in 64 bits."""
    z = 8.0 if Z is None else per_column(Z, N, K, group)
    return (unpack_w4(Q, N, K).double() - z) * per_column(S, N, K, group)
