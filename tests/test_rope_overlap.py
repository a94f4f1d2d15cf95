"""Which outputs of kvs_rotate lie apart from its inputs and from one another, by their addresses and strides alone (no GPU): calls that are
let through end at the launch, which fails without a device."""
import random

import pytest

torch = pytest.importorskip("torch")

INVALID_ARG, CUDA = 1, 2
D = 64
A = 1 << 20                                            # addresses that are never followed
pytestmark = pytest.mark.skipif(torch.cuda.is_available(), reason="the addresses are not real")


@pytest.fixture(scope="module")
def rotate():
    from sparse_kv_cache_decode_gb300 import build as B
    B.build()
    import sparse_kv_cache_decode_gb300 as K
    rope = K.Rope(K.make_rope_config(D))

    def call(n, q, qo, k=None, ko=None):
        """Each (first element, token stride, head stride, heads), in elements."""
        p = lambda x: (A + 2 * x[0], *x[1:3])  # noqa: E731
        k, ko = k or (0, 0, 0, 0), ko or (0, 0, 0, 0)
        return K.lib().kvs_rotate(rope.h, *p(q), q[3], None, *p(qo), *p(k), k[3], None, *p(ko), 4096, 0, n, None)
    return call


FAR = 1 << 22


@pytest.mark.parametrize("n", [1, 2, 3, 41])
def test_rows_between_others(rotate, n):
    """A layout that serves many tokens serves one."""
    h = 8
    row = h * 3 * D                                    # a token's heads, each q, k and v
    part = lambda i: (i * D, row, 3 * D, h)  # noqa: E731
    assert rotate(n, part(0), part(0), part(1), part(1)) == CUDA                                  # q and k in place
    assert rotate(n, part(0), part(2)) == CUDA and rotate(n, part(2), part(0)) == CUDA            # into the columns of v
    assert rotate(n, part(0), part(1), part(2), part(2)) == CUDA
    for i in (0, 1):                                                                              # every second head into the others
        assert rotate(n, (i * D, h * D, 2 * D, h // 2), ((1 - i) * D, h * D, 2 * D, h // 2)) == CUDA
    # [heads][2][tokens]: a head's tokens together
    assert rotate(n, (0, D, 2 * n * D, h), (n * D, D, 2 * n * D, h)) == CUDA
    # one key head between the queries' heads
    assert rotate(n, (0, row, 3 * D, h), (0, row, 3 * D, h), (4 * D, row, D, 1), (5 * D, row, D, 1)) == CUDA
    # those that do meet: the other part's heads, half a head or a head further, q's output over k
    for bad in ((part(0), part(1), part(1), part(1)), (part(0), (D // 2, row, 3 * D, h)), (part(0), (3 * D, row, 3 * D, h)),
                (part(0), (-8, row, 3 * D, h)), (part(0), part(2), part(1), part(2)), ((0, row, 3 * D, h), (2 * D + 8, row, 3 * D, h)),
                (part(0), part(0), (3 * D, row, D, 1), (3 * D, row, D, 1)), (part(0), (3 * (h - 1) * D, row, D, 1)[:3] + (h,)),
                ((0, D, 2 * n * D, h), (n * D - 8, D, 2 * n * D, h))):
        assert rotate(n, *bad) == INVALID_ARG, bad


def elements(n, x):
    p, tok, head, heads = x
    return {p + t * tok + i * head + e for t in range(n) for i in range(heads) for e in range(0, D, 8)}


def test_layouts_at_random(rotate):
    """What is let through lies apart, or is the same; what has the same strides, or is of one token, and lies apart, is let through."""
    r = random.Random(3)
    seen = {True: 0, False: 0}
    for _ in range(6000):
        n, heads = r.choice((1, 1, 2, 3, 5)), r.choice((1, 2, 3, 4))
        unit = r.choice((D, D, D + 8, 2 * D, 3 * D))
        if r.random() < 0.6:                           # a token's heads together
            head = unit * r.choice((1, 1, 2, 3))
            tok = head * heads + r.choice((0, 0, D, unit, 8))
        else:                                          # a head's tokens together
            tok = unit * r.choice((1, 2))
            head = tok * n + r.choice((0, D, tok * n, 8))
        q = (FAR, tok, head, heads)
        at = FAR + r.choice((0, 8, -8, D, -D, head, -head, tok, unit, n * tok, r.randrange(-40, 40) * 8, r.randrange(-40, 40) * D))
        same_strides = r.random() < 0.8
        qo = (at, tok, head, heads) if same_strides else (at, r.choice((tok, head * heads)), r.choice((head, D)), heads)
        if not same_strides and (n > 1 and heads > 1 and qo[1] < (heads - 1) * qo[2] + D and qo[2] < (n - 1) * qo[1] + D):
            continue                                   # its own rows overlap
        got = rotate(n, q, qo)
        meets = bool(elements(n, q) & elements(n, qo))
        same = q[0] == qo[0] and (n == 1 or q[1] == qo[1]) and (heads == 1 or q[2] == qo[2])
        where = (n, q, qo)
        if meets and not same:
            assert got == INVALID_ARG, where
        elif same or n == 1 or (q[1] == qo[1] and (q[2] == qo[2] or heads == 1)):
            assert got == CUDA, where
        seen[got == CUDA] += 1
    assert min(seen.values()) > 500
