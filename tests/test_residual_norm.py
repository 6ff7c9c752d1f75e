"""moe_residual_norm: post-norm, gate, residual scale, residual add and pre-norm
in one pass, against the float64 oracle; its refusals; its place between the
layers of a stack."""
import ctypes

import numpy as np
import pytest
import torch

import sparse_moe_routed_amd as moe
from oracle import moe as om

FAKE = 0x100000  # never dereferenced: the calls below fail validation first


# --------------------------------------------------------------------------- CPU
def test_oracle_closed_forms():
    x = np.zeros((2, 4))
    y = np.array([[3.0, -3.0, 3.0, -3.0], [0.0, 0.0, 0.0, 0.0]])
    # |y| constant: y / rms(y) is its sign; a zero row stays zero (eps > 0)
    xn, out = om.residual_norm(x, y, scale=0.5, eps=0.0 + 1e-30)
    assert np.allclose(xn[0], [0.5, -0.5, 0.5, -0.5]) and np.all(xn[1] == 0) and np.all(out[1] == 0)
    assert np.allclose(out[0], [1, -1, 1, -1])
    # without a post-norm and with gates it is x + s g y; weights scale each channel
    xn, out = om.residual_norm(x + 1, y, gate=np.array([[2.0], [0.0]]), post_norm=False, scale=0.25,
                               pre_weight=np.array([1.0, 2.0, 0.0, 1.0]))
    assert np.allclose(xn[0], [2.5, -0.5, 2.5, -0.5]) and np.allclose(xn[1], 1.0)
    assert np.allclose(out[1], [1, 2, 0, 1], atol=1e-5)


def test_validation():
    f = moe.lib().moe_residual_norm

    def call(T=4, H=64, x=FAKE, y=FAKE + 4096, yd=1, gate=None, kind=0, post=None, pre=None, s=1.0,
             eps=1e-6, pn=1, xo=FAKE, out=FAKE + 8192):
        return f(T, H, x, y, yd, gate, kind, post, pre, s, eps, pn, xo, out, None)

    assert call(T=0, x=None, y=None, xo=None, out=None) == moe.OK
    for bad in (dict(T=-1), dict(T=(1 << 20) + 1), dict(H=0), dict(H=-8), dict(x=None), dict(yd=2),
                dict(kind=4), dict(kind=-1), dict(kind=1), dict(pn=2), dict(eps=-1.0),
                dict(eps=float("nan")), dict(eps=float("inf")), dict(xo=None), dict(xo=FAKE + 4096),
                dict(out=FAKE), dict(out=FAKE + 4096), dict(xo=FAKE + 8192), dict(pn=0, post=FAKE),
                dict(out=None, pre=FAKE), dict(y=None), dict(y=None, xo=None, out=None),
                dict(y=None, xo=None, kind=2), dict(y=None, xo=None, post=FAKE),
                dict(x=FAKE + 1), dict(y=FAKE + 2), dict(yd=0, y=FAKE + 1), dict(xo=FAKE + 1),
                dict(out=FAKE + 3), dict(kind=1, gate=FAKE + 2), dict(post=FAKE + 2),
                dict(pre=FAKE + 1)):
        assert call(**bad) == moe.EINVAL, bad
    assert call(H=49153) == moe.EUNSUPPORTED


# --------------------------------------------------------------------------- GPU
def _close(got, want, m, what):
    """|got - want| within half a bf16 step of want (2^-8 relative, 2^-134 below
    the normal range) and the fp32 steps before it: sums of at most 48 values a
    lane, 6 lane steps and 16 waves are within 70 * 2^-24 of themselves, half
    of that after the root, and 8 more products: 50 * 2^-24 of the term m."""
    tol = 2.0 ** -8 * np.abs(want) + 50 * 2.0 ** -24 * (np.abs(want) + np.abs(m)) + 2.0 ** -134
    bad = np.abs(got - want) > tol
    assert not bad.any(), (what, int(bad.sum()), float(np.abs(got - want)[bad].max()))


def _case(T, H, ydt, kind, seed):
    g = torch.Generator().manual_seed(seed)
    r = lambda *s: torch.randn(s, generator=g)
    x = (2 * r(T, H)).bfloat16()
    y = (0.3 * r(T, H)).to(ydt)
    gate = {"none": None, "token": torch.sigmoid(r(T, 1)), "channel": r(H), "element": torch.sigmoid(r(T, H))}[kind]
    return x, y, gate, 1 + 0.1 * r(H), 1 + 0.1 * r(H)


@pytest.mark.gpu
@pytest.mark.parametrize("T,H,ydt,kind,post,weights", [
    (1, 2688, torch.float32, "channel", True, True),
    (5, 1, torch.float32, "element", True, True),
    (3, 7, torch.bfloat16, "token", True, False),
    (9, 8, torch.float32, "none", False, False),
    (33, 511, torch.bfloat16, "element", True, True),
    (64, 2690, torch.float32, "token", True, True),
    (4, 2689, torch.bfloat16, "channel", False, True),
    (7, 6 * 512 + 1, torch.float32, "channel", True, True),   # first width of four waves
    (3, 4 * 6 * 512 + 5, torch.bfloat16, "element", True, True),  # first of sixteen
    (2, 49152, torch.float32, "channel", True, True),         # widest
    (4096, 192, torch.float32, "token", True, True),
    (1999, 512, torch.bfloat16, "element", True, True),       # the widths and row counts at
    (1536, 513, torch.float32, "none", True, True),           # which a row's waves change
    (1537, 2690, torch.bfloat16, "element", True, True),
    (1537, 6 * 512 + 3, torch.float32, "channel", True, True),
    (5, 8192, torch.bfloat16, "token", True, True),
    (1600, 8191, torch.float32, "channel", False, True),
    (3, 8193, torch.float32, "element", True, True),
    (2, 16385, torch.bfloat16, "channel", True, False),
])
def test_matches_oracle(T, H, ydt, kind, post, weights):
    x, y, gate, pw, rw = _case(T, H, ydt, kind, 7 * T + H)
    d = lambda t: None if t is None else t.cuda()
    xo, out = moe.residual_norm(d(x), d(y), x_out=torch.empty_like(x).cuda(), gate=d(gate),
                                post_weight=d(pw) if post and weights else None,
                                pre_weight=d(rw) if weights else None, scale=0.7, post_norm=post)
    n = lambda t: None if t is None else t.float().numpy().astype(np.float64)
    s = float(np.float32(0.7))
    want, _ = om.residual_norm(n(x), n(y), n(gate), n(pw) if post and weights else None, None, s,
                               float(np.float32(1e-6)), post)
    got = n(xo.cpu())
    _close(got, want, want - n(x), "x'")
    # the pre-norm takes the stored x'
    _, want = om.residual_norm(got, None, pre_weight=n(rw) if weights else None, eps=float(np.float32(1e-6)))
    _close(n(out.cpu()), want, want, "out")


@pytest.mark.gpu
def test_in_place_none_and_first_block():
    x, y, gate, pw, rw = _case(12, 320, torch.float32, "channel", 3)
    x, y, gate, pw, rw = (t.cuda() for t in (x, y, gate, pw, rw))
    xo, out = moe.residual_norm(x, y, x_out=torch.empty_like(x), gate=gate, post_weight=pw, pre_weight=rw)
    x1 = x.clone()
    r, o1 = moe.residual_norm(x1, y, gate=gate, post_weight=pw, pre_weight=rw)
    assert r is x1 and torch.equal(x1, xo) and torch.equal(o1, out)
    x2 = x.clone()
    r, none = moe.residual_norm(x2, y, gate=gate, post_weight=pw, pre_norm=False)
    assert none is None and torch.equal(x2, xo)
    keep = xo.clone()
    same, o3 = moe.residual_norm(xo, None, pre_weight=rw)
    assert same is xo and torch.equal(xo, keep) and torch.equal(o3, out)
    # unit weights and no gate: the same pre-norm as the weightless one, up to one rounding
    _, o4 = moe.residual_norm(xo, None)
    ref = moe.prenorm(xo)
    assert (o4.float() - ref.float()).abs().max() <= 2.0 ** -7 * ref.float().abs().max()
    assert (o4 == ref).float().mean() > 0.99


@pytest.mark.gpu
def test_rows_are_apart_and_nothing_behind_is_written():
    T, H = 6, 333
    x, y, gate, pw, rw = (t.cuda() for t in _case(T, H, torch.float32, "element", 5))
    ref_x, ref_o = moe.residual_norm(x, y, x_out=torch.empty_like(x), gate=gate, post_weight=pw, pre_weight=rw)
    y2 = y.clone()
    y2[2, 5], y2[4, 0] = float("nan"), float("inf")
    store = torch.full((2, T * H + 64), 7.0, dtype=torch.bfloat16, device="cuda")
    bx, bo = store[0, :T * H].view(T, H), store[1, :T * H].view(T, H)
    moe.residual_norm(x, y2, out=bo, x_out=bx, gate=gate, post_weight=pw, pre_weight=rw)
    for t in (0, 1, 3, 5):
        assert torch.equal(bx[t], ref_x[t]) and torch.equal(bo[t], ref_o[t])
    assert bx[2].isnan().all() and bo[2].isnan().all() and bo[4].isnan().any()
    assert (store[:, T * H:] == 7.0).all()
    # no rows: nothing happens
    e = torch.empty((0, H), dtype=torch.bfloat16, device="cuda")
    xo, o = moe.residual_norm(e, torch.empty((0, H), device="cuda"), gate=pw)
    assert o.shape == (0, H)
    # a zero block output and a zero x stay zero
    z = torch.zeros((3, H), dtype=torch.bfloat16, device="cuda")
    xo, o = moe.residual_norm(z, torch.zeros((3, H), device="cuda"))
    assert not xo.any() and not o.any()


@pytest.mark.gpu
def test_refusals_of_the_binding():
    x = torch.zeros((4, 64), dtype=torch.bfloat16, device="cuda")
    y = torch.zeros((4, 64), device="cuda")
    for kw in (dict(y=y.half()), dict(y=y.cpu()), dict(y=y[:3]), dict(y=y, gate=torch.ones(4, device="cuda")),
               dict(y=y, gate=torch.ones(64, device="cuda").bfloat16()), dict(y=y, pre_weight=y[0, :32]),
               dict(y=None, gate=torch.ones(64, device="cuda")), dict(y=y, out=x[:, :32]),
               dict(y=y, out=torch.empty_like(x), pre_norm=False)):
        with pytest.raises(ValueError):
            moe.residual_norm(x, **kw)
    with pytest.raises(ValueError):
        moe.residual_norm(x.float(), y)
    with pytest.raises(ValueError):
        moe.residual_norm(torch.zeros((64, 4), dtype=torch.bfloat16, device="cuda").t(), y)
    with pytest.raises(moe.MoeError):
        moe.residual_norm(x, y, out=x)


@pytest.mark.gpu
def test_stream_and_graph():
    x, y, gate, pw, rw = (t.cuda() for t in _case(17, 2688, torch.float32, "channel", 9))
    want = moe.residual_norm(x, y, x_out=torch.empty_like(x), gate=gate, post_weight=pw, pre_weight=rw)
    xo, out = torch.empty_like(x), torch.empty_like(x)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        moe.residual_norm(x, y, out=out, x_out=xo, gate=gate, post_weight=pw, pre_weight=rw)
    side.synchronize()
    assert torch.equal(xo, want[0]) and torch.equal(out, want[1])
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        moe.residual_norm(x, y, out=out, x_out=xo, gate=gate, post_weight=pw, pre_weight=rw)
    for k in range(3):
        y.mul_(0.5)
        want = moe.residual_norm(x, y, x_out=torch.empty_like(x), gate=gate, post_weight=pw, pre_weight=rw)
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(xo, want[0]) and torch.equal(out, want[1])


def test_overlapping_buffers_are_refused():
    """Rows go to workgroups in any order, so an output that lies over another row's
    input is refused; x_out may be x itself, and neighbours may touch."""
    f = moe.lib().moe_residual_norm
    n = 4 * 64 * 2  # bytes of a bf16 operand

    def call(x=FAKE, y=FAKE + 4096, yd=1, gate=None, kind=0, post=None, pre=None, xo=FAKE, out=FAKE + 8192):
        return f(4, 64, x, y, yd, gate, kind, post, pre, 1.0, 1e-6, 1, xo, out, None)

    for bad in (dict(xo=FAKE + 2), dict(xo=FAKE + n - 2), dict(xo=FAKE - n + 2), dict(xo=FAKE + 4096 + 2),
                dict(xo=FAKE + 4096 + 2 * n - 2), dict(out=FAKE + 128), dict(out=FAKE + 4096 + 2 * n - 2),
                dict(xo=FAKE + 2048, out=FAKE + 2048 + n - 2), dict(y=None, xo=None, out=FAKE + 2),
                dict(kind=1, gate=FAKE + 8192 + 4), dict(kind=2, gate=FAKE + n - 4),
                dict(kind=3, gate=FAKE + 8192 - 2 * n + 4), dict(post=FAKE + n - 4), dict(pre=FAKE + 8192 - 252),
                dict(yd=0, xo=FAKE + 2048, y=FAKE + 2048 + n - 2)):
        assert call(**bad) == moe.EINVAL, bad
