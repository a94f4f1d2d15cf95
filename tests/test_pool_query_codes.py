"""How an E4M3 pool's kernel for few rows holds a row of Q: scaled by a power of two, so that its largest element lies in
[2^7, 2^8), and split into two E4M3 codes that add up.  An element down to 2^-9 of the largest is held exactly, a smaller
one to half a step of the subnormals, 2^-10, which is at most 2^-17 of the largest."""
import numpy as np
import pytest
import torch

from pool_harness import PoolCase

EXACT, BOUND = 2.0 ** -9, 2.0 ** -17
SIGNIFICANDS = torch.arange(128, 256).double() / 128          # all of bf16's


def test_split_arithmetic():
    """Every significand at every exponent, next to the smallest and the largest element that a row's largest may become."""
    code = lambda x: x.float().to(torch.float8_e4m3fn).double()  # noqa: E731
    most = 0.0
    for largest in (128.0, 255.0):
        for e in range(-24, 8):
            x = SIGNIFICANDS * 2.0 ** e
            x = x[x <= largest]
            hi = code(x)
            err = (x - hi - code(x - hi)).abs()
            assert (err <= BOUND * largest).all(), e
            assert (err[x >= EXACT * largest] == 0).all(), e
            most = max(most, float(err.max()) / largest)
    assert most == BOUND                                       # and no smaller bound would do


@pytest.mark.gpu
@pytest.mark.parametrize("row", [2.0 ** -60, 1.0, 2.0 ** 30])
@pytest.mark.parametrize("d", [64, 128])
def test_elements_as_the_kernel_holds_them(d, row):
    """Request j's only key is 1 in dim j and 0 elsewhere, so the log-sum-exp of a row is its element j times the softmax
    scale, which is chosen so that a row's largest element gives a logit of 2^10 to 2^11.  A logit carries the roundings of
    the scale (3), of the product, of log-sum-exp's own sum and of its factor ln 2 (2): 7 * 2^-24 of it, below 2^-21; its weight
    is 2^x of an x that the logit's rounding leaves, so the logarithm of their sum adds as much again and 2^-22 for the exponential."""
    g = 32
    c = PoolCase(d, [1] * (d - 1), [1] * (d - 1), g, 1, d, 16, "fp8", k_scale=1.0, v_scale=1.0)
    one_hot = torch.zeros((d - 1, d), dtype=torch.uint8)
    one_hot[torch.arange(d - 1), torch.arange(1, d)] = 0x38                # 1.0
    c.k[0, torch.from_numpy(c.table[:, 0]).long(), 0, 0] = one_hot
    r = np.random.default_rng(d)
    per = g * (d - 1)
    x = torch.cat([SIGNIFICANDS * 2.0 ** -e for e in range(1, 1 + -(-per // 128))])[:per]
    x = x[torch.from_numpy(r.permutation(per))] * torch.from_numpy(r.choice([-1.0, 1.0], per))
    largest = SIGNIFICANDS[torch.from_numpy(r.integers(0, 128, g))]       # of each row, in dim 0
    rows = torch.cat([largest[:, None], x.view(g, d - 1)], 1) * row
    c.q = rows.to(torch.bfloat16)[None].repeat(d - 1, 1, 1)
    assert torch.equal(c.q[0].double(), rows)
    scale = 2.0 ** 10 / row
    c.cuda(softmax_scale=scale)
    out, lse = c.out()
    c.pool.attn(0, c.d_q, c.d_cu, c.d_ctx, c.d_table, out, lse=lse)
    assert c.pool.poll_error() == 0
    got, want = lse.double().cpu().T, rows[:, 1:] * scale                  # [row][element]
    tol = 2.0 ** -20 * want.abs() + 2.0 ** -21
    tol = torch.where(rows[:, 1:].abs() >= EXACT * rows[:, :1], tol, tol + BOUND * rows[:, :1] * scale)
    off = (got - want).abs()
    assert (off <= tol).all(), float((off / tol).max())
