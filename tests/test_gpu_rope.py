"""Norms and rotation of query and key rows, dense and into a pool, and kept keys at new positions, against fp64.

Tolerance of a rotated element y of a pair of length M (the oracle's mag): the norm's sum of squares is of 16 products a lane and a few
sums across lanes, its root and the weight's product take 4 more roundings: 12 * 2^-24 relative at most (the root halves the sum's).  The angle is
rounded to 2^-24 turns (2^-21.3), its product with 2 pi by pi * 2^-24 (2^-22.3), and off by the position times 2^-53 (2^-22 at 2^31); its cosine and
sine are off by 2^-21 at most; two products and a sum: 3 * 2^-24.  Together below 2^-18 M.  Then one rounding: half a step of bf16, 2^-8 |y|, or of E4M3, 2^-4 |y| or 2^-10 of the
code's unit below its normal range."""
import numpy as np
import pytest
import torch

import sparse_kv_cache_decode_gb300 as K
from oracle import rope_freqs, rope_rows

pytestmark = pytest.mark.gpu
BAD_INDEX = 7


def bf16(r, *shape, scale=1.0):
    return torch.from_numpy((r.standard_normal(shape) * scale).astype(np.float32)).to(torch.bfloat16).cuda()


def f64(t):
    return t.double().cpu().numpy()


def check(got, want, mag, where=""):
    tol = 2.0 ** -8 * np.abs(want) + 2.0 ** -18 * mag + 1e-38
    err = np.abs(f64(got) - want)
    assert (err <= tol).all(), f"{where}: off by {(err / tol).max():.2f} of the tolerance"


def check_codes(codes, want, mag, scale):
    """E4M3 codes (uint8) of want / scale."""
    got = codes.view(torch.float8_e4m3fn).double().cpu().numpy()
    w = np.clip(want / scale, -448, 448)
    tol = 2.0 ** -4 * np.abs(w) + 2.0 ** -10 + 2.0 ** -18 * mag / scale
    assert (np.abs(got - w) <= tol).all()


def weight(r, d):
    return torch.from_numpy((1 + 0.3 * r.standard_normal(d)).astype(np.float32)).cuda()


class Case:
    def __init__(self, seed, n, hq, hk, d, rot=None, theta=1e4, adjacent=False, sections=None, cycle=False, norm=True, far=1 << 20, eps=1e-6, scale=1.0):
        r = self.rng = np.random.default_rng(seed)
        self.n, self.hq, self.hk, self.d, self.eps, self.scale, self.adjacent = n, hq, hk, d, eps, scale, adjacent
        self.rot = d if rot is None else rot
        self.axes = None if sections is None else K.rope_axes(sections, cycle)
        self.freqs = rope_freqs(self.rot, theta)
        self.rope = K.Rope(K.make_rope_config(d, self.rot, theta=theta, adjacent=adjacent, axes=self.axes, rot_scale=scale, norm_eps=eps))
        self.pos = torch.from_numpy(r.integers(-far, far, (self.rope.n_axis, n)).astype(np.int32)).cuda()
        self.q, self.k = bf16(r, n, hq, d, scale=2.0), bf16(r, n, hk, d)
        self.wq, self.wk = (weight(r, d), weight(r, d)) if norm else (None, None)

    def ref(self, x, w):
        return rope_rows(f64(x), self.pos.cpu().numpy(), self.freqs, self.axes, self.adjacent, None if w is None else f64(w), self.eps, self.scale)

    def rotate(self, **kw):
        qo, ko = torch.full_like(self.q, 7.0), torch.full_like(self.k, 7.0)
        if self.hk == 0:
            self.rope.rotate(self.q, self.pos, qo, q_norm=self.wq, **kw)
            return qo, ko
        self.rope.rotate(self.q, self.pos, qo, self.k, ko, q_norm=self.wq, k_norm=self.wk, **kw)
        return qo, ko

    def check(self, qo, ko):
        check(qo, *self.ref(self.q, self.wq), "q")
        check(ko, *self.ref(self.k, self.wk), "k")


@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("adjacent", [False, True])
@pytest.mark.parametrize("n,hq,hk", [(1, 32, 8), (5, 7, 1), (77, 1, 1), (300, 12, 3), (6000, 3, 2), (1701, 11, 5), (20001, 0, 3), (4567, 17, 0)])
def test_dense(d, adjacent, n, hq, hk):
    c = Case(n + d, n, hq, hk, d, adjacent=adjacent)
    c.check(*c.rotate())


@pytest.mark.parametrize("d,rot,adjacent", [(64, 64, False), (64, 48, True), (128, 128, False), (128, 96, False), (256, 256, True)])
def test_a_row_does_not_depend_on_the_others(d, rot, adjacent):
    """A prompt in one call, in chunks and token by token gives the same bits."""
    c = Case(50, 3001, 9, 3, d, rot=rot, adjacent=adjacent, sections=[rot // 4, rot // 4])
    whole = c.rotate()
    qo, ko = torch.zeros_like(c.q), torch.zeros_like(c.k)
    at = [0, 1, 2, 39, 500, 501, 3001]
    for a, b in zip(at, at[1:]):
        c.rope.rotate(c.q[a:b], c.pos[:, a:b].contiguous(), qo[a:b], c.k[a:b], ko[a:b], q_norm=c.wq, k_norm=c.wk)
    assert torch.equal(qo, whole[0]) and torch.equal(ko, whole[1])


@pytest.mark.parametrize("d,rot", [(64, 0), (64, 16), (64, 48), (128, 16), (128, 64), (128, 96), (128, 112), (256, 64), (256, 144)])
@pytest.mark.parametrize("adjacent", [False, True])
@pytest.mark.parametrize("norm", [False, True])
def test_part_of_a_row_turns(d, rot, adjacent, norm):
    c = Case(rot, 37, 5, 3, d, rot=rot, adjacent=adjacent, norm=norm, scale=1.25)
    qo, ko = c.rotate()
    c.check(qo, ko)
    if not norm:
        assert torch.equal(qo[..., rot:], c.q[..., rot:]) and torch.equal(ko[..., rot:], c.k[..., rot:])


@pytest.mark.parametrize("sections,cycle", [([16, 24, 24], False), ([22, 21, 21], True), ([8] * 8, True), ([0, 64], False)])
@pytest.mark.parametrize("adjacent", [False, True])
@pytest.mark.parametrize("n", [1, 130])
def test_several_axes(sections, cycle, adjacent, n):
    c = Case(3, n, 9, 2, 128, sections=sections, cycle=cycle, adjacent=adjacent)
    c.check(*c.rotate())
    one = c.pos[0].contiguous()                     # the same position on all axes: any of them, given once
    c.pos = one.expand(c.rope.n_axis, n).contiguous()
    whole = c.rotate()
    c.check(*whole)
    qo, ko = torch.empty_like(c.q), torch.empty_like(c.k)
    c.rope.rotate(c.q, one, qo, c.k, ko, q_norm=c.wq, k_norm=c.wk)
    assert torch.equal(qo, whole[0]) and torch.equal(ko, whole[1])
    wide = torch.full((c.rope.n_axis, n + 5), 77, dtype=torch.int32, device="cuda")       # a part of longer rows of positions
    wide[:, 3:n + 3] = c.pos
    qo.zero_()
    c.rope.rotate(c.q, wide[:, 3:n + 3], qo, q_norm=c.wq)
    assert torch.equal(qo, whole[0])


@pytest.mark.parametrize("far", [1, 1 << 24, (1 << 31) - 1])
def test_far_positions(far):
    c = Case(far % 97, 64, 4, 2, 128, theta=5e5, far=far, norm=False)
    c.pos[0, 0], c.pos[0, 1] = far, -far
    c.check(*c.rotate())


def test_frequencies_of_ones_own():
    c = Case(5, 50, 4, 2, 64)
    c.freqs = np.concatenate([np.linspace(-2.0, 9.0, 31), [0.0]])
    c.rope = K.Rope(K.make_rope_config(64, inv_freq=c.freqs, norm_eps=c.eps))
    c.check(*c.rotate())
    # half a turn a position, either way: exactly one sign
    rope = K.Rope(K.make_rope_config(64, inv_freq=[np.pi] * 16 + [-np.pi] * 16))
    out = torch.empty_like(c.q)
    rope.rotate(c.q, torch.full((50,), 1 << 20, dtype=torch.int32, device="cuda"), out)
    assert torch.equal(out, c.q)
    rope.rotate(c.q, torch.full((50,), -7, dtype=torch.int32, device="cuda"), out)
    assert torch.equal(out, -c.q)


def test_strided_rows_and_in_place():
    c = Case(8, 41, 6, 2, 64, adjacent=True)
    qo, ko = c.rotate()
    # a fused projection, in place: the rest of it stays
    x = bf16(c.rng, 41, 12, 64)
    x[:, 1:7], x[:, 8:10] = c.q, c.k
    before = x.clone()
    c.rope.rotate(x[:, 1:7], c.pos, x[:, 1:7], x[:, 8:10], x[:, 8:10], q_norm=c.wq, k_norm=c.wk)
    before[:, 1:7], before[:, 8:10] = qo, ko
    assert torch.equal(x, before)
    # the last dims of longer rows, and every second head
    y, z = bf16(c.rng, 41, 6, 96), bf16(c.rng, 41, 4, 64)
    y[:, :, 32:], z[:, ::2] = c.q, c.k
    before = y.clone(), z.clone()
    c.rope.rotate(y[:, :, 32:], c.pos, y[:, :, 32:], z[:, ::2], z[:, 1::2], q_norm=c.wq, k_norm=c.wk)
    before[0][:, :, 32:], before[1][:, 1::2] = qo, ko
    assert torch.equal(y, before[0]) and torch.equal(z, before[1])
    # a batch of which every second token is taken
    w = bf16(c.rng, 82, 6, 64)
    w[::2] = c.q
    out = torch.empty_like(c.q)
    c.rope.rotate(w[::2], c.pos, out, q_norm=c.wq)
    assert torch.equal(out, qo)
    # a head's tokens together
    t = torch.empty((6, 41, 64), dtype=torch.bfloat16, device="cuda")
    c.rope.rotate(c.q, c.pos, t.transpose(0, 1), q_norm=c.wq)
    assert torch.equal(t.transpose(0, 1), qo)
    with pytest.raises(K.KvsError):
        c.rope.rotate(w[:41], c.pos, w[1:42])
    with pytest.raises(K.KvsError):
        c.rope.rotate(w.view(-1)[4:4 + 41 * 384].view(41, 6, 64), c.pos, out)


def test_rows_of_zeros_infinities_and_nan_stay_by_themselves():
    c = Case(9, 10, 4, 2, 128)
    c.q[2, 1], c.q[3, 0, 5], c.q[4, 2, 7], c.k[5, 1] = 0, float("inf"), float("nan"), 0
    qo, ko = c.rotate()
    assert (qo[2, 1] == 0).all() and (ko[5, 1] == 0).all()
    ok = torch.ones((10, 4), dtype=torch.bool)
    ok[3, 0] = ok[4, 2] = False
    with np.errstate(invalid="ignore"):
        want, mag = c.ref(c.q, c.wq)
    got = f64(qo)[ok.numpy()]
    assert (np.abs(got - want[ok.numpy()]) <= 2.0 ** -8 * np.abs(want[ok.numpy()]) + 2.0 ** -18 * mag[ok.numpy()]).all()
    assert not torch.isfinite(qo[4, 2]).any() and not torch.isfinite(qo[3, 0, [5, 69]]).any()
    # without an eps a row of zeros has no norm
    c.rope = K.Rope(K.make_rope_config(128, norm_eps=0.0))
    c.eps = 0.0
    qo, _ = c.rotate()
    check(qo[:2], *(a[:2] for a in c.ref(c.q, c.wq)))


@pytest.mark.parametrize("n", [20, 9000])
@pytest.mark.parametrize("adjacent", [False, True])
def test_elements_that_do_not_turn_stay_by_themselves(n, adjacent):
    c = Case(15, n, 3, 1, 128, rot=32, norm=False, adjacent=adjacent)
    for i, x in ((40, float("inf")), (41, float("nan")), (127, -float("inf")), (96, float("nan"))):
        c.q[i % n, 1, i] = x
    qo, _ = c.rotate()
    assert torch.equal(qo[..., 32:].view(torch.int16)[torch.isfinite(c.q[..., 32:])], c.q[..., 32:].view(torch.int16)[torch.isfinite(c.q[..., 32:])])
    assert torch.equal(torch.isnan(qo), torch.isnan(c.q)) and torch.equal(torch.isinf(qo), torch.isinf(c.q))
    check(qo[..., :32], *(a[..., :32] for a in c.ref(c.q, None)))


def test_no_tokens_and_no_keys():
    c = Case(10, 4, 4, 2, 64)
    e = c.q[:0]
    c.rope.rotate(e, c.pos[:, :0], e, c.k[:0], c.k[:0])
    out = torch.empty_like(c.q)
    c.rope.rotate(c.q, c.pos, out)
    check(out, *c.ref(c.q, None))
    for a, kw in [((c.q, c.pos[:, :3], out), {}), ((c.q, c.pos.long(), out), {}), ((c.q, c.pos, out[:3]), {}), ((c.q, c.pos, out.float()), {}),
                  ((c.q, c.pos, out, c.k), {}), ((c.q, c.pos, out, c.k[:3], c.k[:3]), {}), ((c.q, c.pos, out), dict(q_norm=torch.ones(32).cuda())),
                  ((c.q, c.pos.cpu(), out), {}), ((c.q, c.pos, out.cpu()), {})]:
        with pytest.raises(ValueError):
            c.rope.rotate(*a, **kw)


def test_other_streams_and_graphs():
    """Two graphs with the same handle, replayed beside an eager call on a third stream."""
    cases = [Case(20 + i, 200 + i, 8, 2, 128) for i in range(3)]
    want = [c.rotate() for c in cases]
    outs = [(torch.zeros_like(c.q), torch.zeros_like(c.k)) for c in cases]
    streams = [torch.cuda.Stream() for _ in cases]
    graphs = []
    rope = cases[0].rope
    torch.cuda.synchronize()
    for c, o, s in list(zip(cases, outs, streams))[:2]:
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=s):
            rope.rotate(c.q, c.pos, o[0], c.k, o[1], q_norm=c.wq, k_norm=c.wk)
        graphs.append(g)
    for _ in range(2):
        for o in outs:
            o[0].zero_()
            o[1].zero_()
        torch.cuda.synchronize()
        for g, s in zip(graphs, streams):
            with torch.cuda.stream(s):
                g.replay()
        c, o = cases[2], outs[2]
        rope.rotate(c.q, c.pos, o[0], c.k, o[1], q_norm=c.wq, k_norm=c.wk, stream=streams[2])
        torch.cuda.synchronize()
        for o, w in zip(outs, want):
            assert torch.equal(o[0], w[0]) and torch.equal(o[1], w[1])


# ------------------------------------------------------------------ into a pool
class PoolRows(Case):
    def __init__(self, seed, n, hq, hk, d, bs=16, kv="bf16", spare=3, n_layer=1, **kw):
        super().__init__(seed, n, hq, hk, d, **kw)
        self.bs, self.kv = bs, kv
        self.scales = (0.05, 0.03) if kv == "fp8" else (1.0, 1.0)
        self.n_slots = -(-n // bs) + spare
        shape = (n_layer, self.n_slots, hk, bs, d)
        t = torch.float8_e4m3fn if kv == "fp8" else torch.bfloat16
        self.kp, self.vp = (torch.full(shape, float("nan"), device="cuda").to(t) for _ in range(2))
        self.v = bf16(self.rng, n, hk, d)
        self.pool = K.Pool(K.make_pool_config(n_layer, self.n_slots, hq, hk, d, bs, self.n_slots * bs, 4, max(n, 1), kv_dtype=kv,
                                              k_scale=self.scales[0], v_scale=self.scales[1]), self.kp, self.vp)
        self.place = torch.from_numpy(self.rng.permutation(self.n_slots * bs)[:n].astype(np.int64)).cuda()

    def go(self, layer=0, q_out=None, **kw):
        qo = torch.full_like(self.q, 7.0) if q_out is None else q_out
        self.pool.rotate_append(layer, self.rope, self.q, self.k, self.v, self.pos, self.place, qo, q_norm=self.wq, k_norm=self.wk, **kw)
        return qo

    def rows(self, pool, layer=0):
        """[places][H_kv][d] as patterns."""
        x = pool[layer].view(torch.uint8 if self.kv == "fp8" else torch.int16)
        return x.transpose(1, 2).reshape(-1, self.hk, self.d)


@pytest.mark.parametrize("kv", ["bf16", "fp8"])
@pytest.mark.parametrize("d,adjacent,rot,sections", [(128, False, None, None), (64, True, None, None), (128, False, 96, [16, 16, 16]), (64, False, 16, None),
                                                     (128, True, 32, [8, 8])])
@pytest.mark.parametrize("n,hq,hk,bs", [(1, 32, 8, 16), (33, 7, 7, 128), (500, 9, 3, 32), (5000, 4, 2, 64), (1301, 15, 5, 16)])
def test_append(kv, d, adjacent, rot, sections, n, hq, hk, bs):
    c = PoolRows(n + d, n, hq, hk, d, bs, kv, adjacent=adjacent, rot=rot, sections=sections)
    if n > 2:
        c.place[n // 2] = -1                        # a token without a place
    qo = c.go()
    dense_q, dense_k = c.rotate()
    assert torch.equal(qo, dense_q)
    kr, vr = c.rows(c.kp), c.rows(c.vp)
    ok = c.place >= 0
    at = c.place[ok]
    if kv == "bf16":
        assert torch.equal(kr[at], dense_k[ok].view(torch.int16)) and torch.equal(vr[at], c.v[ok].view(torch.int16))
    else:
        want, mag = c.ref(c.k[ok], c.wk) if bool(ok.all()) else (a[ok.cpu().numpy()] for a in c.ref(c.k, c.wk))
        check_codes(kr[at], want, mag, c.scales[0])
        codes = torch.empty(int(ok.sum()) * hk * d, dtype=torch.uint8, device="cuda")
        K.quantize_e4m3(c.v[ok].contiguous().view(-1), codes, c.scales[1])
        assert torch.equal(vr[at].reshape(-1), codes)
    rest = torch.ones(kr.shape[0], dtype=torch.bool, device="cuda")
    rest[at] = False
    nan = torch.full((1,), float("nan"), device="cuda").to(c.kp.dtype).view(kr.dtype).item()
    assert (kr[rest] == nan).all() and (vr[rest] == nan).all()
    assert c.pool.poll_error() == 0


def test_append_as_pool_append_does():
    """Without norm or rotation the two appends write the same."""
    for kv in ("bf16", "fp8"):
        c = PoolRows(4, 40, 4, 2, 64, kv=kv, rot=0, norm=False)
        table = torch.arange(c.n_slots, dtype=torch.int32, device="cuda").flip(0).view(1, -1).contiguous()
        cu, ctx = (torch.tensor(x, dtype=torch.int32, device="cuda") for x in ([0, 40], [53]))
        pos = torch.empty(40, dtype=torch.int32, device="cuda")
        c.pool.places(cu, ctx, table, c.place, pos)
        assert pos.tolist() == list(range(13, 53))
        c.go()
        got = c.rows(c.kp).clone(), c.rows(c.vp).clone()
        c.kp.view(torch.uint8).fill_(255), c.vp.view(torch.uint8).fill_(255)
        c.pool.append(0, c.k, c.v, cu, ctx, table)
        at = c.place
        assert torch.equal(got[0][at], c.rows(c.kp)[at]) and torch.equal(got[1][at], c.rows(c.vp)[at])


@pytest.mark.parametrize("scale", [1.0, 0.05, 0.0625, 0.3333333, 1.9999999, 1e-3, 7.77e5, 3.0 * 2.0 ** -61, 2.0 ** -60, 2.0 ** 60, 1.5 * 2.0 ** 61, 1e-38, 3e38])
def test_every_value_is_quantised_as_the_quantiser_does(scale):
    """All bf16 patterns (infinities and NaN among them) as V rows of an E4M3 pool."""
    hk, d, bs = 8, 128, 16
    n = 65536 // (hk * d)
    kp, vp = (torch.zeros((1, n // bs, hk, bs, d), dtype=torch.uint8, device="cuda") for _ in range(2))
    pool = K.Pool(K.make_pool_config(1, n // bs, hk, hk, d, bs, n, 1, n, kv_dtype="fp8", k_scale=scale, v_scale=scale), kp, vp)
    v = torch.arange(-32768, 32768, dtype=torch.int32, device="cuda").to(torch.int16).view(torch.bfloat16).view(n, hk, d)
    q = torch.zeros_like(v)
    place = torch.arange(n, device="cuda")
    pool.rotate_append(0, K.Rope(K.make_rope_config(d, rot_dim=0)), q, v, v.clone(), torch.zeros(n, dtype=torch.int32, device="cuda"), place, q.clone())
    codes = torch.empty(65536, dtype=torch.uint8, device="cuda")
    K.quantize_e4m3(v.view(-1), codes, scale)
    for p in (vp, kp):                              # K, neither normed nor rotated, is the same values
        got = p[0].transpose(1, 2).reshape(-1)
        assert torch.equal(got, codes), (got != codes).nonzero()[:5]


def test_append_layers_and_strides():
    c = PoolRows(6, 30, 6, 2, 128, n_layer=3, norm=True)
    want = c.go(layer=0)
    x = bf16(c.rng, 30, 11, 128)
    x[:, :6], x[:, 6:8], x[:, 9:] = c.q, c.k, c.v
    rest = x[:, 6:].clone()
    c.q, c.k, c.v = x[:, :6], x[:, 6:8], x[:, 9:]
    c.go(layer=2, q_out=c.q)                        # q in place in the fused projection
    assert torch.equal(c.q, want) and torch.equal(x[:, 6:], rest)
    for p in (c.kp, c.vp):
        assert torch.equal(p[0].view(torch.int16), p[2].view(torch.int16)) and torch.isnan(p[1]).all()
    for bad in (3, -1):
        with pytest.raises(K.KvsError):
            c.go(layer=bad)
    with pytest.raises(K.KvsError):
        c.go(q_out=x[:, 3:9])                       # over k
    with pytest.raises(K.KvsError):
        c.go(q_out=x[:, 5:])                        # over k and v
    other = K.Rope(K.make_rope_config(64))
    with pytest.raises(K.KvsError):
        c.pool.rotate_append(0, other, c.q, c.k, c.v, c.pos, c.place, c.q)
    many = torch.zeros((31, 6, 128), dtype=torch.bfloat16, device="cuda")
    kv = many[:, :2].contiguous()
    with pytest.raises(K.KvsError):
        c.pool.rotate_append(0, c.rope, many, kv, kv.clone(), torch.zeros(31, dtype=torch.int32, device="cuda"),
                             torch.arange(31, device="cuda"), many)
    e = c.q[:0]
    c.pool.rotate_append(0, c.rope, e, c.k[:0], c.v[:0], c.pos[:, :0], c.place[:0], e)
    assert c.pool.poll_error() == 0


def test_places_outside_the_pool():
    c = PoolRows(7, 20, 4, 2, 64)
    end = c.n_slots * c.bs
    c.place[3], c.place[5], c.place[7], c.place[9] = end, (1 << 62), -(1 << 62), -2
    qo = c.go()
    assert c.pool.poll_error() == BAD_INDEX and c.pool.poll_error() == 0
    assert torch.equal(qo, c.rotate()[0])
    ok = (c.place >= 0) & (c.place < end)
    assert torch.equal(c.rows(c.kp)[c.place[ok]], c.rotate()[1][ok].view(torch.int16))
    c.place[3], c.place[5] = -1, -1
    c.go()
    assert c.pool.poll_error() == 0


@pytest.mark.parametrize("kv", ["bf16", "fp8"])
def test_rows_behind_the_fourth_gigabyte(kv):
    """A pool whose last rows lie past 2^32 bytes: append there, then reposition them."""
    hk, bs, d = 8, 128, 128
    n_slots = 18000 if kv == "bf16" else 36000
    kind = torch.float8_e4m3fn if kv == "fp8" else torch.bfloat16
    kp, vp = (torch.zeros((1, n_slots, hk, bs, d), dtype=kind, device="cuda") for _ in range(2))
    assert kp.numel() * kp.element_size() > 1 << 32
    pool = K.Pool(K.make_pool_config(1, n_slots, hk, hk, d, bs, 3 * bs, 1, 300, kv_dtype=kv), kp, vp)
    c = Case(30, 300, hk, hk, d)
    table = torch.tensor([[n_slots - 1, 0, n_slots - 2]], dtype=torch.int32, device="cuda")
    v = bf16(c.rng, 300, hk, d)
    place, qo = torch.empty(300, dtype=torch.int64, device="cuda"), torch.empty_like(c.q)
    cu, ctx = (torch.tensor(x, dtype=torch.int32, device="cuda") for x in ([0, 300], [300]))
    pool.places(cu, ctx, table, place)
    pool.rotate_append(0, c.rope, c.q, c.k, v, c.pos, place, qo, q_norm=c.wq, k_norm=c.wk)
    rows = lambda p: p[0][table[0].long()].transpose(1, 2).reshape(-1, hk, d)[:300]  # noqa: E731
    want, mag = c.ref(c.k, c.wk)
    check(rows(kp).to(torch.bfloat16), want, mag) if kv == "bf16" else check_codes(rows(kp).view(torch.uint8), want, mag, 1.0)
    assert torch.equal(rows(vp).float(), v.float().clamp(-448, 448).to(kind).float())
    before = f64(rows(kp).float())
    kept = torch.arange(300, dtype=torch.int32, device="cuda").add_(7).expand(1, hk, 300).contiguous()
    pool.reposition(0, c.rope, kept, ctx, table)
    y, mag = rope_rows(before, np.full((1, 300), -7), c.freqs)
    half = (2.0 ** -4 * np.abs(y) + 2.0 ** -10) if kv == "fp8" else 2.0 ** -8 * np.abs(y)
    assert (np.abs(f64(rows(kp).float()) - y) <= half + 2.0 ** -18 * mag).all()
    assert not kp[0, 1:n_slots - 2].view(torch.uint8).any() and not vp[0, 1:n_slots - 2].view(torch.uint8).any()
    assert pool.poll_error() == 0


def test_a_captured_step():
    """Tables, rotation and append in one graph, replayed with other lengths and rows, beside the same calls one by one."""
    n_req, hq, hk, d, bs = 4, 8, 2, 64, 16
    r = np.random.default_rng(40)
    sets = []
    for _ in range(2):
        kp, vp = (torch.zeros((1, 40, hk, bs, d), dtype=torch.bfloat16, device="cuda") for _ in range(2))
        pool = K.Pool(K.make_pool_config(1, 40, hq, hk, d, bs, 128, n_req, 8), kp, vp)
        sets.append((pool, K.BlockTables.empty(pool, n_req), kp, vp, torch.empty(8, dtype=torch.int64, device="cuda"),
                     torch.empty(8, dtype=torch.int32, device="cuda"), torch.empty((8, hq, d), dtype=torch.bfloat16, device="cuda")))
    rope = K.Rope(K.make_rope_config(d))
    x = bf16(r, 8, hq + 2 * hk, d)
    cu, ctx = (torch.tensor(a, dtype=torch.int32, device="cuda") for a in ([0, 2, 4, 6, 8], [0] * 4))

    def step(pool, tables, kp, vp, place, pos, qo):
        tables.reserve(ctx, cu, place, pos)
        pool.rotate_append(0, rope, x[:, :hq], x[:, hq:hq + hk], x[:, hq + hk:], pos, place, qo)

    ctx.fill_(2)
    for s in sets:
        step(*s)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        step(*sets[0])
    for i in range(9):
        ctx.add_(2 if i != 4 else -3)
        x.copy_(bf16(r, 8, hq + 2 * hk, d))
        g.replay()
        step(*sets[1])
        for a, b in zip(sets[0][2:], sets[1][2:]):
            assert torch.equal(a, b)
        assert torch.equal(sets[0][1].n_held, sets[1][1].n_held) and torch.equal(sets[0][1].ring_state, sets[1][1].ring_state)
    assert sets[0][0].poll_error() == 0 and sets[1][0].poll_error() == 0


# ------------------------------------------------------------------ kept keys
@pytest.mark.parametrize("kv", ["bf16", "fp8"])
@pytest.mark.parametrize("d,adjacent,rot", [(128, False, 128), (64, True, 64), (64, False, 48), (128, True, 16), (128, False, 0)])
@pytest.mark.parametrize("keep,bs,hk", [(1, 16, 3), (37, 16, 2), (300, 64, 1)])
def test_reposition(kv, d, adjacent, rot, keep, bs, hk):
    r = np.random.default_rng(keep + d)
    n_kept = [keep, 0, max(0, keep - 5), min(1, keep)]
    nb = -(-keep // bs) + 1
    n_slots = 4 * nb + 2
    kind = torch.float8_e4m3fn if kv == "fp8" else torch.bfloat16
    kp = bf16(r, 1, n_slots, hk, bs, d, scale=100.0 if kv == "fp8" else 1.0).float().clamp(-440, 440).to(kind)
    pool = K.Pool(K.make_pool_config(1, n_slots, hk, hk, d, bs, nb * bs, 4, 8, kv_dtype=kv, k_scale=0.1), kp, torch.zeros_like(kp.float()).to(kind))
    table = torch.from_numpy(r.permutation(n_slots)[:4 * nb].reshape(4, nb).astype(np.int32)).cuda()
    kept = np.full((4, hk, keep), -9, np.int32)
    for i, m in enumerate(n_kept):
        for h in range(hk):
            kept[i, h, :m] = np.sort(r.choice(70000, m, replace=False))
    kept[0, 0, 0] = 0                               # stays where it is
    if keep > 200:                                  # far away, on either side, and where the sums change
        kept[2, 0, :9] = [(1 << 31) - 1, -(1 << 31) + 9, (1 << 24) + 1, -(1 << 24), (1 << 22) + 3, (1 << 22) + 5, 5 - (1 << 22), 7 - (1 << 22), 1 << 30]
    rope = K.Rope(K.make_rope_config(d, rot, theta=5e5, adjacent=adjacent, rot_scale=1.5))
    before = kp.clone()
    pool.reposition(0, rope, torch.from_numpy(kept).cuda(), torch.tensor(n_kept, dtype=torch.int32, device="cuda"), table)
    assert pool.poll_error() == 0
    freqs = rope_freqs(rot, 5e5)
    want, tol, touched = f64(before.float()), np.zeros(kp.shape), np.zeros(kp.shape, bool)
    for i, m in enumerate(n_kept):
        slot = table[i].cpu().numpy()[np.arange(m) // bs]
        for h in range(hk):
            x = want[0, slot, h, np.arange(m) % bs]
            y, mag = rope_rows(x[:, None], (np.arange(m) - kept[i, h, :m].astype(np.int64))[:, None], freqs, adjacent=adjacent)
            y, mag = y[:, 0], mag[:, 0]
            if kv == "fp8":
                y = np.clip(y, -448, 448)
            want[0, slot, h, np.arange(m) % bs] = y
            tol[0, slot, h, np.arange(m) % bs] = (2.0 ** -4 * np.abs(y) + 2.0 ** -10 if kv == "fp8" else 2.0 ** -8 * np.abs(y)) + 2.0 ** -18 * mag
    got = f64(kp.float())
    assert (np.abs(got - want) <= tol).all()        # tol 0: rows that are not kept, as they were


def test_reposition_refuses_and_reports():
    r = np.random.default_rng(0)
    kp = bf16(r, 1, 6, 2, 16, 64)
    pool = K.Pool(K.make_pool_config(1, 6, 4, 2, 64, 16, 32, 2, 8), kp, torch.zeros_like(kp))
    i32 = lambda x: torch.tensor(x, dtype=torch.int32, device="cuda")  # noqa: E731
    kept = torch.full((2, 2, 20), 5, dtype=torch.int32, device="cuda")
    table = i32([[0, 1], [2, 3]])
    rope = K.Rope(K.make_rope_config(64))
    for bad in (K.Rope(K.make_rope_config(64, axes=[0, 1] * 16)), K.Rope(K.make_rope_config(128))):
        with pytest.raises(K.KvsError):
            pool.reposition(0, bad, kept, i32([20, 20]), table)
    with pytest.raises(K.KvsError):
        pool.reposition(0, rope, torch.zeros((2, 2, 33), dtype=torch.int32, device="cuda"), i32([20, 20]), table)
    with pytest.raises(K.KvsError):
        pool.reposition(1, rope, kept, i32([20, 20]), table)
    assert pool.poll_error() == 0
    for n, t in ((i32([20, 21]), table), (i32([20, -1]), table), (i32([20, 20]), i32([[0, 1], [6, -1]]))):
        before = kp.clone()
        pool.reposition(0, rope, kept, n, t)
        assert pool.poll_error() == BAD_INDEX
        assert torch.equal(kp[:, 2:], before[:, 2:]) and not torch.equal(kp[:, :2], before[:, :2])
