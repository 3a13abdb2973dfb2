"""Inputs under which every row's share of the cross entropy gradients' sums is visible.

All logits of a residual row are equal, so that D = h / V everywhere (no loss gradient: labels
outside the vocabulary), and h is V times a power of two: in 16 bits D is that power exactly (it
is off by less than 1e-5 of it before its rounding).  Three blocks of columns:
  column 0           x = 1, table = 1: the logits
  the first half     x = 0, table = whole numbers: d_residual there is D times the table's column sums
  the second half    x = whole numbers, table = 0: d_table there is the same in each row, the sum of D x
The numbers are positive and so few bits wide that every partial sum in f32 is exact: 16-bit results
have to be the rounded exact ones.  Where D is f32 (f32 tables; up to 8 residual rows and n V row bytes
of 128 MiB) they are within D's error and the sums'.
"""
import torch

from tests.training_labels import half_step


def make(n, V, d, dtype, device="cpu", seed=0):
    """(E, x, labels, h): D is 2^-(8 + b % 3) for row b."""
    gen = torch.Generator(device=device).manual_seed(seed + n + V + d)
    half = d // 2
    E = torch.zeros((V, d), dtype=dtype, device=device)
    E[:, 0] = 1
    step = max(1, (1 << 27) // d)
    for v in range(0, V, step):  # 1 .. 3, or 1 where 3 V would not fit 24 bits less D's 2
        rows = min(step, V - v)
        top = 4 if V < 1 << 20 else 2
        E[v:v + rows, 1:half] = torch.randint(1, top, (rows, half - 1), generator=gen, device=device,
                                              dtype=torch.int8).to(dtype)
    x = torch.zeros((n, d), dtype=dtype, device=device)
    x[:, 0] = 1
    x[:, half:] = torch.randint(1, 8, (n, d - half), generator=gen, device=device, dtype=torch.int8).to(dtype)
    labels = torch.full((n,), -1, dtype=torch.int32, device=device)
    D = torch.tensor([2.0 ** -8, 2.0 ** -9, 2.0 ** -10], dtype=torch.float64, device=device)[torch.arange(n) % 3]
    return E, x, labels, (D * V).float()


def want(E, x, h):
    """(dx in the first half, dE's row in the second), before their rounding."""
    V, d = E.shape
    half = d // 2
    D = (h.double().cpu() / V).to(E.device)  # (on a device, division by a number may be a product with its inverse)
    sums = torch.zeros(half - 1, dtype=torch.float64, device=E.device)
    step = max(1, (1 << 27) // d)
    for v in range(0, V, step):
        sums += E[v:v + step, 1:half].double().sum(0)
    return D[:, None] * sums[None, :], (D[:, None] * x[:, half:].double()).sum(0)


def one_pass(n, V, d, dtype):
    """Up to 8 rows and 128 MiB of table reads: D is f32 and both gradients come from one pass over the table."""
    return n <= 8 and n * V * d * (4 if dtype == torch.float32 else 2) <= 128 << 20


def exact_d(n, V, d, dtype):
    """Whether D is rounded to 16 bits: a power of two then."""
    return dtype != torch.float32 and not one_pass(n, V, d, dtype)


def bound(v, n, V, d, dtype):
    """D a power of two: the result's rounding alone.  Else D is off by less than 1e-5 of itself, and the sums
    round: V terms of a matrix core's accumulator by 2^-22 each at most (n > 8), or, one pass over the
    table, about 2,048 waves' V / 2,048 rows per KiB of a row, and the join of their sums."""
    if exact_d(n, V, d, dtype):
        return half_step(v, dtype)
    size = 4 if dtype == torch.float32 else 2
    waves = max(16, V * -(-d * size // 1024) // 2048 + 1) + 2048 // 16 + 16
    chain = waves if one_pass(n, V, d, dtype) else V + 64
    return v.abs() * (1e-5 + chain * 2.0 ** -22) + half_step(v, dtype)


# the kernels of both products: one pass, 64, 128 and 256 columns, K slices, several pieces, tables whose
# last tile is partial, more tiles than workgroups
CASES = [("bf16", 8, 40001, 64), ("f32", 4, 70001, 64), ("f16", 3, 100001, 128), ("f32", 8, 20001, 1000),
         ("bf16", 8, 150001, 128), ("f16", 8, 300003, 64), ("bf16", 20, 3001, 264), ("bf16", 64, 100001, 256),
         ("f16", 65, 30000, 264), ("bf16", 100, 20011, 328), ("bf16", 128, 40001, 264), ("f32", 40, 30001, 132),
         ("f32", 300, 9001, 600), ("f32", 600, 24003, 524), ("bf16", 300, 151936, 136), ("bf16", 700, 40001, 520),
         ("f16", 700, 20001, 520), ("bf16", 40000, 9000, 64)]
TYPES = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}
