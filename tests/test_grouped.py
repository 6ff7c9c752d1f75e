"""Products of bf16 rows grouped by expert and their gradients against float64, the
grouping of rows, autograd, refusals."""
import numpy as np
import pytest
import torch

import sparse_moe_routed_amd as moe

FAKE = 0x100000  # never dereferenced: the calls below fail validation first


# --------------------------------------------------------------------------- CPU
def test_validation():
    L = moe.lib()
    a, w, o, y = (FAKE + (i << 24) for i in range(4))  # 16 MiB apart
    for fn, width in ((L.moe_grouped_matmul, (64, 128)), (L.moe_grouped_input_grad, (128, 64))):
        def call(R=40, E=4, N=64, K=128, a=a, w=w, o=o, y=y, yd=0, z=0):
            return fn(R, E, N, K, a, w, o, y, yd, z, None)

        for bad in (dict(R=-1), dict(E=0), dict(N=0), dict(K=-8), dict(a=None), dict(w=None), dict(o=None),
                    dict(y=None), dict(a=a + 8), dict(w=w + 2), dict(o=o + 2), dict(y=y + 4), dict(yd=2),
                    dict(z=2), dict(z=-1)):
            assert call(**bad) == moe.EINVAL, bad
        for bad in (dict(E=257), dict(N=60), dict(K=130), dict(N=65544), dict(K=65544), dict(R=(1 << 23) + 1)):
            assert call(**bad) == moe.EUNSUPPORTED, bad
        assert call(R=0, a=None, y=None) == moe.OK and call(R=0, yd=5) == moe.EINVAL
        out, rows = width  # the output's columns and the operand's
        for yd, size in ((0, 2), (1, 4)):
            for bad in (a, a + 40 * rows * 2 - 16, w + 4 * 64 * 128 * 2 - 16, o - 40 * out * size + 16, o):
                assert call(y=bad, yd=yd) == moe.EINVAL, hex(bad)

    def dw(R=40, E=4, N=64, K=128, dy=a, x=w, o=o, dw=y, d=0, acc=0, ws=None, nb=0):
        return L.moe_grouped_weight_grad(R, E, N, K, dy, x, o, dw, d, acc, ws, nb, None)

    for bad in (dict(R=-1), dict(E=0), dict(dy=None), dict(x=None), dict(o=None), dict(dw=None), dict(dy=a + 8),
                dict(x=w + 8), dict(o=o + 1), dict(dw=y + 8), dict(d=2), dict(acc=2), dict(acc=1),
                dict(dw=a + 40 * 64 * 2 - 16), dict(dw=w), dict(dw=o), dict(R=0, dw=None)):
        assert dw(**bad) == moe.EINVAL, bad
    for bad in (dict(E=257), dict(N=60), dict(K=130), dict(R=(1 << 23) + 1)):
        assert dw(**bad) == moe.EUNSUPPORTED, bad
    assert dw(R=0, dy=None, x=None, d=1, acc=1) == moe.OK  # nothing to add
    # parts of the rows where the matrices are few and small
    size = L.moe_grouped_weight_grad_workspace_size
    assert size(40, 4, 64, 128) == 256 and size(24576, 128, 1856, 2688) == 256 and size(40, 4, 60, 128) == 0
    need = size(8192, 1, 64, 128)
    assert need > 256 and (need - 256) % (64 * 128 * 4) == 0
    big, ws = dict(R=8192, E=1), FAKE + (5 << 24)
    for bad in (dict(), dict(ws=ws, nb=need - 1), dict(ws=ws + 16, nb=need)):
        assert dw(**big, **bad) == moe.EWORKSPACE, bad
    for bad in (a, a + 8192 * 128 - 256, w, y, o - need + 256):
        assert dw(**big, ws=bad, nb=need) == moe.EINVAL, hex(bad)


def test_validation_of_group_rows():
    L = moe.lib()
    need = L.moe_group_rows_workspace_size(128, 5000)
    assert need > 0 and need % 256 == 0 and L.moe_group_rows_workspace_size(128, 0) > 0
    for bad in ((0, 5), (257, 5), (4, -1), (4, (1 << 23) + 1)):
        assert L.moe_group_rows_workspace_size(*bad) == 0
    i, o, s, v, ws = (FAKE + (k << 20) for k in range(5))

    def call(R=5000, E=128, i=i, o=o, s=s, v=v, ws=ws, nb=need):
        return L.moe_group_rows(R, E, i, o, s, v, ws, nb, None)

    for bad in (dict(R=-1), dict(E=0), dict(i=None), dict(o=None), dict(s=None), dict(v=None), dict(i=i + 2),
                dict(o=o + 1), dict(s=s + 2), dict(v=v + 3), dict(o=i), dict(s=i + 19996), dict(v=s), dict(v=i + 4),
                dict(i=ws + 256), dict(o=ws + 512)):
        assert call(**bad) == moe.EINVAL, bad
    for bad in (dict(E=257), dict(R=(1 << 23) + 1)):
        assert call(**bad) == moe.EUNSUPPORTED, bad
    for bad in (dict(ws=None), dict(nb=need - 1), dict(ws=ws + 16)):
        assert call(**bad) == moe.EWORKSPACE, bad


# --------------------------------------------------------------------------- GPU
def _counts(kind, E, R, seed):
    """Rows of each expert, R in all."""
    rng = np.random.default_rng(seed)
    if kind == "even":
        return np.full(E, R // E) + (np.arange(E) < R % E)
    if kind == "one":  # everything at one expert, the others empty
        c = np.zeros(E, int)
        c[E // 2] = R
        return c
    share = rng.permutation(np.arange(1, E + 1)) ** -1.0 * (rng.random(E) < 0.7)
    share[rng.integers(E)] = 1.0
    return rng.multinomial(R, share / share.sum())


class Case:
    def __init__(self, kind, R, E, N, K, rest=0, seed=0):
        g = torch.Generator().manual_seed(seed + R + N)
        self.R, self.E, self.N, self.K, self.rows = R + rest, E, N, K, R
        self.bounds = np.concatenate([[0], np.cumsum(_counts(kind, E, R, seed))])
        self.x = torch.randn((self.R, K), generator=g).bfloat16()
        self.dy = torch.randn((self.R, N), generator=g).bfloat16()
        self.w = (torch.randn((E, N, K), generator=g) / K ** 0.5).bfloat16()
        self.off = torch.from_numpy(self.bounds).int().cuda()

    def cuda(self):
        return self.x.cuda(), self.dy.cuda(), self.w.cuda(), self.off

    def ref(self, op, *tensors):
        """float64 result of `op`, and the same of the operands' magnitudes."""
        out = []
        for f in (lambda t: t.double(), lambda t: t.double().abs()):
            x, dy, w = f(self.x), f(self.dy), f(self.w)
            shape = {"y": (self.R, self.N), "dx": (self.R, self.K), "dw": (self.E, self.N, self.K)}[op]
            r = torch.zeros(shape, dtype=torch.float64)
            for e in range(self.E):
                s = slice(self.bounds[e], self.bounds[e + 1])
                if op == "y":
                    r[s] = x[s] @ w[e].T
                elif op == "dx":
                    r[s] = dy[s] @ w[e]
                else:
                    r[e] = dy[s].T @ x[s]
            out.append(r)
        return out

    def terms(self, op):
        return {"y": self.K, "dx": self.N, "dw": int(np.diff(self.bounds).max())}[op]


def _check(got, ref, size, terms, base=None):
    """An fp32 sum of n exact products in any order is off by at most n roundings (or
    cuts, 2^-23) of the sum of their magnitudes; a result in bf16 by half a step
    (2^-8) more, and below the normal range by 2^-134.  In the mean n roundings of
    partial sums that grow like sqrt(n) come to sqrt(n / 6) 2^-23 of the result's size
    (twice that is allowed), that to bf16 to at most 2.26e-3 (2.4e-3)."""
    half = 2.0 ** -8 if got.dtype == torch.bfloat16 else 2.0 ** -24
    err = (got.double().cpu() - ref).abs()
    assert torch.isfinite(got).all()
    bound = (terms + 1) * 2.0 ** -23 * (size + (0 if base is None else base)) + half * ref.abs() + 2.0 ** -134
    assert (err <= bound).all(), float((err / bound).max())
    if ref.numel() >= 4096 and float(ref.norm()) > 0:
        mean = 2 * (terms / 6) ** 0.5 * 2.0 ** -23 + (2.4e-3 if got.dtype == torch.bfloat16 else 2.0 ** -23)
        assert err.norm() <= mean * ref.norm()


SHAPES = [
    ("even", 1, 1, 8, 8, 0), ("one", 1, 5, 64, 64, 3), ("even", 3, 2, 72, 136, 0), ("skew", 24, 128, 192, 320, 0),
    ("skew", 100, 16, 136, 72, 20), ("skew", 300, 7, 200, 264, 300), ("one", 257, 3, 128, 128, 1),
    ("even", 511, 1, 1000, 200, 0), ("skew", 700, 256, 64, 96, 5), ("even", 1000, 4, 512, 1024, 0),
    ("skew", 2500, 16, 320, 192, 77), ("one", 1300, 256, 256, 384, 0), ("skew", 4000, 3, 1856, 88, 0),
    ("skew", 6000, 8, 264, 1352, 130), ("skew", 5, 16, 1000, 392, 0), ("skew", 40, 3, 200, 1352, 9),
    ("even", 64, 1, 72, 2688, 0), ("one", 8000, 1, 64, 72, 0), ("skew", 9001, 2, 136, 264, 5),
    ("one", 5000, 3, 256, 128, 0), ("skew", 5200, 3, 2056, 72, 30), ("skew", 5200, 3, 72, 2056, 30),
    ("skew", 5200, 20, 136, 2056, 30), ("skew", 700, 16, 2056, 104, 9), ("one", 700, 16, 1856, 136, 0),
    ("skew", 6000, 4, 1000, 1800, 0), ("even", 24001, 1, 360, 368, 0),
    ("skew", 2600, 3, 1856, 104, 7),
]


@pytest.mark.gpu
@pytest.mark.parametrize("kind,R,E,N,K,rest", SHAPES)
def test_products(kind, R, E, N, K, rest):
    c = Case(kind, R, E, N, K, rest)
    x, dy, w, off = c.cuda()
    calls = {"y": (lambda **kw: moe.grouped_matmul(x, w, off, **kw), (c.R, N)),
             "dx": (lambda **kw: moe.grouped_input_grad(dy, w, off, **kw), (c.R, K)),
             "dw": (lambda **kw: moe.grouped_weight_grad(dy, x, off, **kw), (E, N, K))}
    for op, (call, shape) in calls.items():
        ref, size = c.ref(op)
        for dt in (torch.bfloat16, torch.float32):
            n = int(np.prod(shape))
            store = torch.full((n + 1024,), 7.0, dtype=dt, device="cuda")
            out = store[512:512 + n].view(shape)
            call(**{op: out})
            live = out if op == "dw" else out[:R]
            _check(live, ref if op == "dw" else ref[:R], size if op == "dw" else size[:R], c.terms(op))
            # nothing around the output, and no row of no expert, is written
            assert (store[:512] == 7.0).all() and (store[512 + n:] == 7.0).all()
            assert op == "dw" or (out[R:] == 7.0).all()
            again = call(**{op + "_dtype": dt})
            assert torch.equal(again if op == "dw" else again[:R], live)
            assert op == "dw" or not again[R:].any()
        if op == "dw":
            empty = np.nonzero(np.diff(c.bounds) == 0)[0]
            assert not again[empty].any()
            # added to what is there: one fp32 rounding of the sum
            base = torch.randn(shape, generator=torch.Generator().manual_seed(1))
            total = moe.grouped_weight_grad(dy, x, off, dw=base.cuda(), accumulate=True)
            assert torch.equal(total, again + base.cuda())


@pytest.mark.gpu
@pytest.mark.parametrize("R", [24, 3000, 4000])
def test_full_layer_sizes(R):
    """The layer's own widths with its uneven use of 128 experts; every result of a few
    experts, one bit for bit the same each time."""
    g = torch.Generator().manual_seed(R)
    E, N, K = 128, 1856, 2688
    c = _counts("skew", E, R, R)
    b = np.concatenate([[0], np.cumsum(c)])
    x, dy = (torch.randn((R, n), generator=g).bfloat16() for n in (K, N))
    w = torch.empty((E, N, K), dtype=torch.bfloat16, device="cuda").normal_(0, K ** -0.5)
    off = torch.from_numpy(b).int().cuda()
    y, dx = moe.grouped_matmul(x.cuda(), w, off), moe.grouped_input_grad(dy.cuda(), w, off)
    dw = moe.grouped_weight_grad(dy.cuda(), x.cuda(), off)
    used = np.nonzero(c)[0]
    for e in {used[0], used[-1], int(np.argmax(c))}:
        s, we = slice(b[e], b[e + 1]), w[e].cpu().double()
        xs, ds = x[s].double(), dy[s].double()
        _check(y[s], xs @ we.T, xs.abs() @ we.abs().T, K)
        _check(dx[s], ds @ we, ds.abs() @ we.abs(), N)
        _check(dw[e], ds.T @ xs, ds.abs().T @ xs.abs(), c[e])
    assert torch.equal(moe.grouped_matmul(x.cuda(), w, off), y)
    assert torch.equal(moe.grouped_input_grad(dy.cuda(), w, off), dx)
    assert torch.equal(moe.grouped_weight_grad(dy.cuda(), x.cuda(), off), dw)
    assert not dw[np.nonzero(c == 0)[0]].any()


@pytest.mark.gpu
@pytest.mark.parametrize("R", [60, 2000])
def test_rows_and_experts_are_apart(R):
    """NaN and infinity in a row, in an expert's weight and in rows of no expert."""
    c = Case("even", R, 5, 136, 264, rest=9)
    x, dy, w, off = c.cuda()
    y, dx, dw = (moe.grouped_matmul(x, w, off), moe.grouped_input_grad(dy, w, off),
                 moe.grouped_weight_grad(dy, x, off))
    per = R // 5
    r = 2 * per + 1  # a row of expert 2
    x2, dy2, w2 = x.clone(), dy.clone(), w.clone()
    x2[r, 3] = float("nan")
    dy2[r, 130] = float("inf")
    x2[R:], dy2[R:] = float("nan"), float("inf")
    w2[4, 135, 263] = float("nan")
    keep = [i for i in range(R) if i != r and i < 4 * per]
    y2 = moe.grouped_matmul(x2, w2, off)
    assert torch.equal(y2[keep], y[keep]) and y2[r].isnan().all() and not y2[R:].any()
    assert y2[4 * per:R, 135].isnan().all() and torch.equal(y2[4 * per:R, :135], y[4 * per:R, :135])
    dx2 = moe.grouped_input_grad(dy2, w2, off)
    assert torch.equal(dx2[keep], dx[keep]) and not dx2[r].isfinite().any()
    assert dx2[4 * per:R, 263].isnan().all() and torch.equal(dx2[4 * per:R, :263], dx[4 * per:R, :263])
    dw2 = moe.grouped_weight_grad(dy2, x2, off)
    others = [0, 1, 3, 4]
    assert torch.equal(dw2[others], dw[others])
    assert dw2[2][:, 3].isnan().all() and not dw2[2][130].isfinite().any()
    cols, rows = [k for k in range(264) if k != 3], [n for n in range(136) if n != 130]
    assert torch.equal(dw2[2][rows][:, cols], dw[2][rows][:, cols])


@pytest.mark.gpu
def test_rows_past_32_bits():
    """x and dx of 5 GB: the rows behind 2^31 values, and dw's sum over them."""
    R, E, N, K = 40000, 2, 64, 65536
    b = [0, 39000, 39900]  # 100 rows of no expert
    x = torch.empty((R, K), dtype=torch.bfloat16, device="cuda").normal_()
    dy = torch.empty((R, N), dtype=torch.bfloat16, device="cuda").normal_()
    w = torch.empty((E, N, K), dtype=torch.bfloat16, device="cuda").normal_()
    off = torch.tensor(b, dtype=torch.int32, device="cuda")
    y, dx, dw = (moe.grouped_matmul(x, w, off), moe.grouped_input_grad(dy, w, off),
                 moe.grouped_weight_grad(dy, x, off, dw_dtype=torch.float32))
    for e, s in ((0, slice(38980, 39000)), (1, slice(39880, 39900))):
        xs, ds, we = x[s].cpu().double(), dy[s].cpu().double(), w[e].cpu().double()
        _check(y[s], xs @ we.T, xs.abs() @ we.abs().T, K)
        _check(dx[s], ds @ we, ds.abs() @ we.abs(), N)
    xs, ds = x[b[1]:b[2], -512:].cpu().double(), dy[b[1]:b[2]].cpu().double()
    _check(dw[1, :, -512:], ds.T @ xs, ds.abs().T @ xs.abs(), b[2] - b[1])
    assert not y[b[2]:].any() and not dx[b[2]:].any()


@pytest.mark.gpu
def test_weights_past_32_bits():
    """Two matrices of 5 GB: the last rows and columns of either, and of its gradient."""
    R, E, N, K = 100, 2, 65536, 40000
    b = [0, 30, 100]
    x = torch.empty((R, K), dtype=torch.bfloat16, device="cuda").normal_()
    dy = torch.empty((R, N), dtype=torch.bfloat16, device="cuda").normal_()
    w = torch.empty((E, N, K), dtype=torch.bfloat16, device="cuda").normal_()
    off = torch.tensor(b, dtype=torch.int32, device="cuda")
    y, dx, dw = (moe.grouped_matmul(x, w, off), moe.grouped_input_grad(dy, w, off),
                 moe.grouped_weight_grad(dy, x, off))
    for e in range(E):
        s = slice(b[e], b[e + 1])
        xs, ds = x[s].cpu().double(), dy[s].cpu().double()
        last = w[e, -200:].cpu().double()
        _check(y[s, -200:], xs @ last.T, xs.abs() @ last.abs().T, K)
        last = w[e, :, -24:].cpu().double()
        _check(dx[s, -24:], ds @ last, ds.abs() @ last.abs(), N)
        xs, ds = xs[:, -300:], ds[:, -300:]
        _check(dw[e, -300:, -300:], ds.T @ xs, ds.abs().T @ xs.abs(), b[e + 1] - b[e])


@pytest.mark.gpu
def test_no_rows():
    w = torch.randn((3, 64, 128), device="cuda").bfloat16()
    off = torch.zeros(4, dtype=torch.int32, device="cuda")
    x, dy = (torch.empty((0, n), dtype=torch.bfloat16, device="cuda") for n in (128, 64))
    assert moe.grouped_matmul(x, w, off).shape == (0, 64)
    assert moe.grouped_input_grad(dy, w, off).shape == (0, 128)
    assert not moe.grouped_weight_grad(dy, x, off).any()
    keep = torch.ones((3, 64, 128), device="cuda")
    assert (moe.grouped_weight_grad(dy, x, off, dw=keep, accumulate=True) == 1).all()
    # rows, none of which is an expert's
    x, dy = (torch.ones((70, n), dtype=torch.bfloat16, device="cuda") for n in (128, 64))
    y = torch.full((70, 64), 3.0, dtype=torch.bfloat16, device="cuda")
    assert (moe.grouped_matmul(x, w, off, y=y) == 3).all() and not moe.grouped_matmul(x, w, off).any()
    assert not moe.grouped_input_grad(dy, w, off).any() and not moe.grouped_weight_grad(dy, x, off).any()


@pytest.mark.gpu
def test_bounds_that_are_none():
    """Offsets that run backwards or leave the rows: as the header takes them, and
    nothing around the outputs is touched."""
    c = Case("even", 200, 4, 64, 128)
    x, dy, w, _ = c.cuda()
    for bad, groups in (([-9, 50, 300, 300, 2 ** 31 - 1], [(0, 50), (50, 200), (200, 200), (200, 200)]),
                        ([10, 60, 40, 100, -3], [(10, 60), (60, 40), (40, 100), (100, 0)])):
        off = torch.tensor(bad, dtype=torch.int32, device="cuda")
        store = torch.full((200 * 64 + 1024,), 7.0, device="cuda")
        y = moe.grouped_matmul(x, w, off, y=store[512:512 + 200 * 64].view(200, 64))
        assert (store[:512] == 7).all() and (store[-512:] == 7).all()
        dw = moe.grouped_weight_grad(dy, x, off, dw_dtype=torch.float32)
        for e, (a, b) in enumerate(groups):
            s = slice(a, max(a, b))
            _check(dw[e], (c.dy[s].double().T @ c.x[s].double()),
                   (c.dy[s].double().abs().T @ c.x[s].double().abs()), 200)
            if bad[0] == -9 and b > a:
                _check(y[s], c.x[s].double() @ c.w[e].double().T, c.x[s].double().abs() @ c.w[e].double().abs().T, 128)


@pytest.mark.gpu
@pytest.mark.parametrize("T,k,E", [(1, 1, 1), (3, 2, 5), (64, 6, 128), (400, 6, 128), (700, 8, 256), (1000, 3, 16)])
def test_group_rows(T, k, E):
    rng = np.random.default_rng(T)
    ids = rng.integers(0, E, (T, k)).astype(np.int32)
    for drop in (False, True):
        if drop:
            ids[rng.random((T, k)) < 0.2] = E
            ids[rng.random((T, k)) < 0.1] = -1
        off, src, inv = moe.group_rows(torch.from_numpy(ids).cuda(), E)
        flat = ids.reshape(-1)
        live = np.nonzero((flat >= 0) & (flat < E))[0]
        order = live[np.argsort(flat[live], kind="stable")]
        want = np.concatenate([[0], np.cumsum(np.bincount(flat[live], minlength=E))])
        assert np.array_equal(off.cpu().numpy(), want)
        assert np.array_equal(src.cpu().numpy()[:len(order)], order) and not src[len(order):].any()
        back = np.full(T * k, -1)
        back[order] = np.arange(len(order))
        assert inv.shape == (T, k) and np.array_equal(inv.cpu().numpy().reshape(-1), back)
    off, src, inv = moe.group_rows(torch.empty((0, k), dtype=torch.int32, device="cuda"), E)
    assert not off.any() and src.shape == (0,) and inv.shape == (0, k)


@pytest.mark.gpu
def test_refusals_of_the_binding():
    c = Case("even", 20, 2, 64, 128)
    x, dy, w, off = c.cuda()
    e = lambda *shape, dtype=torch.bfloat16: torch.empty(shape, dtype=dtype, device="cuda")
    for bad in (lambda: moe.grouped_matmul(x.float(), w, off), lambda: moe.grouped_matmul(x.cpu(), w, off),
                lambda: moe.grouped_matmul(x[:, :64], w, off), lambda: moe.grouped_matmul(x[0], w, off),
                lambda: moe.grouped_matmul(x, w[0], off), lambda: moe.grouped_matmul(x, w.float(), off),
                lambda: moe.grouped_matmul(x, w.transpose(1, 2), off), lambda: moe.grouped_matmul(dy, w, off),
                lambda: moe.grouped_matmul(x, w, off[:2]), lambda: moe.grouped_matmul(x, w, off.long()),
                lambda: moe.grouped_matmul(x, w, off.cpu()), lambda: moe.grouped_matmul(x, w, off, y=e(20, 63)),
                lambda: moe.grouped_matmul(x, w, off, y=e(20, 64, dtype=torch.float16)),
                lambda: moe.grouped_matmul(x, w, off, y=e(20, 64), y_dtype=torch.float32),
                lambda: moe.grouped_input_grad(x, w, off), lambda: moe.grouped_input_grad(dy, w, off, dx=e(20, 64)),
                lambda: moe.grouped_weight_grad(dy, x[:10], off), lambda: moe.grouped_weight_grad(dy, x, off[:1]),
                lambda: moe.grouped_weight_grad(dy, x, off, accumulate=True),
                lambda: moe.grouped_weight_grad(dy, x, off, dw=e(2, 64, 64)),
                lambda: moe.grouped_weight_grad(dy.t(), x, off),
                lambda: moe.group_rows(torch.zeros(4, device="cuda"), 4), lambda: moe.group_rows(off, 300),
                lambda: moe.group_rows([1, 2], 4)):
        with pytest.raises(ValueError):
            bad()
    with pytest.raises(moe.MoeError) as err:
        moe.grouped_weight_grad(dy, x, off, dw=e(2, 64, 128), accumulate=True)  # bf16 does not accumulate
    assert err.value.status == moe.EINVAL
    with pytest.raises(moe.MoeError) as err:
        moe.grouped_matmul(e(4, 12), e(2, 64, 12), off)
    assert err.value.status == moe.EUNSUPPORTED


@pytest.mark.gpu
@pytest.mark.parametrize("R", [40, 1500])
def test_captured_and_on_two_streams(R):
    c = Case("skew", R, 16, 192, 320, rest=8)
    x, dy, w, off = c.cuda()

    def step(x, dy, off, y, dx, dw):
        moe.grouped_matmul(x, w, off, y=y)
        moe.grouped_input_grad(dy, w, off, dx=dx)
        moe.grouped_weight_grad(dy, x, off, dw=dw, accumulate=True)

    def outs():
        return [torch.zeros((c.R, 192), dtype=torch.bfloat16, device="cuda"),
                torch.zeros((c.R, 320), dtype=torch.bfloat16, device="cuda"), torch.zeros((16, 192, 320), device="cuda")]

    o = outs()
    step(x, dy, off, *o)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        step(x, dy, off, *o)
    for k in range(4):  # other rows at other experts
        d = Case("skew", R, 16, 192, 320, rest=8, seed=10 + k)
        x.copy_(d.x)
        dy.copy_(d.dy)
        off.copy_(d.off)
        want = outs()
        step(x, dy, off, *want)
        for t in o:
            t.zero_()
        g.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(p, q) for p, q in zip(o, want))
    streams = [torch.cuda.Stream() for _ in range(2)]
    both = [outs() for _ in streams]
    torch.cuda.synchronize()
    for s, p in zip(streams, both):
        with torch.cuda.stream(s):
            step(x, dy, off, *p)
    torch.cuda.synchronize()
    assert all(torch.equal(p, q) for b in both for p, q in zip(b, want))


def _experts(h, ids, gates, up, down, linear, group):
    """Experts with a SiLU in place of the layer's ReLU^2."""
    off, src, inv = group(ids, up.shape[0])
    T, k = ids.shape
    a = torch.nn.functional.silu(linear(h[src.long() // k], up, off))
    o = linear(a, down, off)[inv.long()]  # [T, k, H]
    return (o.float() * gates.unsqueeze(2)).sum(1)


@pytest.mark.gpu
@pytest.mark.parametrize("T", [1, 50, 500])
def test_training_step(T):
    """Router, grouping, both projections, another activation and the combine, with the
    gradients of tokens, gates and weights against float64 autograd on the CPU of
    the same formula."""
    H, F, E, k = 128, 192, 16, 3
    d = moe.LayerDims(H, F, E, k)
    g = torch.Generator().manual_seed(T)
    h = torch.randn((T, H), generator=g).bfloat16()
    up = (torch.randn((E, F, H), generator=g) / H ** 0.5).bfloat16()
    down = (torch.randn((E, H, F), generator=g) / F ** 0.5).bfloat16()
    router = moe.pack_router((0.1 * torch.randn((E, H), generator=g)).cuda(), None, d)
    ids, gates = moe.route(h.cuda(), router, d)
    dout = torch.randn((T, H), generator=g)

    leaves = [t.cuda().requires_grad_() for t in (h, gates, up, down)]
    y = _experts(leaves[0], ids, leaves[1], leaves[2], leaves[3], moe.grouped_linear, moe.group_rows)
    got = torch.autograd.grad(y, leaves, dout.cuda())

    def group(ids, E):
        flat = ids.reshape(-1)
        src = torch.argsort(flat, stable=True)
        inv = torch.empty_like(src)
        inv[src] = torch.arange(len(src))
        off = torch.zeros(E + 1, dtype=torch.long)
        off[1:] = torch.bincount(flat, minlength=E).cumsum(0)
        return off, src, inv.view(ids.shape)

    def linear(x, w, off):
        return torch.cat([x[off[e]:off[e + 1]] @ w[e].T for e in range(E)])

    ref_leaves = [t.detach().double().cpu().requires_grad_() for t in leaves]

    def silu_experts(h, gates, up, down):
        off, src, inv = group(ids.cpu().long(), E)
        a = torch.nn.functional.silu(linear(h[src // k], up, off))
        return (linear(a, down, off)[inv] * gates.unsqueeze(2)).sum(1)

    ref = silu_experts(*ref_leaves)
    want = torch.autograd.grad(ref, ref_leaves, dout.double())
    # bf16 after each of the few steps between: h, a, o and their gradients, each off
    # by 2^-8 of itself at most and 1.7e-3 in the mean; six of them in a row stay below
    # six times that
    assert (y.detach().double().cpu() - ref).norm() <= 6 * 2.4e-3 * ref.norm()
    for a, b, t in zip(got, want, leaves):
        assert a.dtype == t.dtype and a.shape == t.shape
        assert (a.double().cpu() - b).norm() <= 6 * 2.4e-3 * b.norm()
    used = torch.bincount(ids.reshape(-1), minlength=E) > 0
    assert not got[2][~used].any() and not got[3][~used].any()


@pytest.mark.gpu
def test_gradients_against_differences():
    """The products are linear in each operand, so a step of any length along a
    direction changes <y, v> by exactly its slope: <dx, dir> and <dw, dir>."""
    c = Case("skew", 300, 8, 64, 128, seed=3)
    x, dy, w, off = c.cuda()
    x, w = x.requires_grad_(), w.requires_grad_()
    dx, dw = torch.autograd.grad(moe.grouped_linear(x, w, off), (x, w), dy)
    g = torch.Generator().manual_seed(5)
    for t, grad in ((x, dx), (w, dw)):
        dir = torch.randn(t.shape, generator=g).bfloat16().cuda()
        f = lambda v: moe.grouped_matmul(v if t is x else x.detach(), v if t is w else w.detach(), off,
                                         y_dtype=torch.float32)
        # dir alone is the difference quotient of a linear function; fp32 outputs
        slope = (f(dir).double() * dy.double()).sum()
        want = (grad.double() * dir.double()).sum()
        # grad is in bf16: each of its values is off by half a step, independent signs
        room = 2.0 ** -8 * (grad.double() * dir.double()).norm() * 6
        assert abs(slope - want) <= room
    # only what is asked for, and a gradient that comes as a view
    xg, = torch.autograd.grad(moe.grouped_linear(x, w.detach(), off).t(), (x,), dy.t())
    assert torch.equal(xg, dx)
    wg, = torch.autograd.grad(moe.grouped_linear(x.detach(), w, off), (w,), dy.t().contiguous().t())
    assert torch.equal(wg, dw)


def _stale(*shape):
    """The allocator's next block of this size holds NaN."""
    torch.full(shape, float("nan"), dtype=torch.bfloat16, device="cuda")


@pytest.mark.gpu
@pytest.mark.parametrize("R,lo,hi", [(40, 2, 5), (40, 0, 3), (40, 5, 8), (1500, 3, 4), (3000, 1, 8), (1500, 4, 4)])
def test_rows_before_the_first_expert(R, lo, hi):
    """Some of the experts, as a process that holds experts lo to hi has them: all rows and
    the bounds of its own.  A new output is zero in the others' rows on both sides, one
    that is given keeps them."""
    c = Case("skew", R, 8, 192, 320, rest=5)
    x, dy, w, off = c.cuda()
    some, own = off[lo:hi + 1].contiguous(), w[lo:hi].contiguous()
    if lo == hi:  # one expert without rows, somewhere inside
        some, own = off[lo].repeat(2), w[lo:lo + 1].contiguous()
    a, b = int(c.bounds[lo]), int(c.bounds[hi])
    grads = []
    for call, rows, width, op in ((moe.grouped_matmul, x, 192, "y"), (moe.grouped_input_grad, dy, 320, "dx")):
        ref, size = c.ref(op)
        _stale(c.R, width)
        new = call(rows, own, some)
        assert not new[:a].any() and not new[b:].any()
        _check(new[a:b], ref[a:b], size[a:b], c.terms(op))
        kept = call(rows, own, some, **{op: torch.full_like(new, 7.0)})
        assert (kept[:a] == 7).all() and (kept[b:] == 7).all() and torch.equal(kept[a:b], new[a:b])
        grads.append(new)
    xl, wl = x.clone().requires_grad_(), own.clone().requires_grad_()
    _stale(c.R, 192)
    y = moe.grouped_linear(xl, wl, some)
    assert torch.equal(y, grads[0])
    _stale(c.R, 320)
    dx, dw = torch.autograd.grad(y, (xl, wl), dy)
    assert torch.equal(dx, grads[1])
    if lo == hi:
        assert not dw.any()
    else:
        ref, size = c.ref("dw")
        _check(dw, ref[lo:hi], size[lo:hi], c.terms("dw"))


@pytest.mark.gpu
def test_bounds_past_the_rows_leave_nothing_stale():
    """All bounds behind the rows, or before them: no row is an expert's."""
    x = torch.ones((300, 64), dtype=torch.bfloat16, device="cuda")
    w = torch.ones((2, 64, 64), dtype=torch.bfloat16, device="cuda")
    for bad in ([300, 300, 300], [400, 500, 600], [-5, -5, -1]):
        off = torch.tensor(bad, dtype=torch.int32, device="cuda")
        for call in (moe.grouped_matmul, moe.grouped_input_grad):
            _stale(300, 64)
            assert not call(x, w, off).any()


@pytest.mark.gpu
@pytest.mark.parametrize("R", [7, 300])
def test_gradient_that_begins_anywhere(R):
    """autograd hands on views: here the part of a longer gradient that begins at its
    fourth value, six bytes in, contiguous and so not copied by contiguous()."""
    c = Case("skew", R, 4, 64, 128)
    x, dy, w, off = c.cuda()
    x, w = x.requires_grad_(), w.requires_grad_()
    head = torch.zeros(3, dtype=torch.bfloat16, device="cuda")
    both = torch.cat([head, moe.grouped_linear(x, w, off).reshape(-1)])
    dx, dw = torch.autograd.grad(both, (x, w), torch.cat([head, dy.reshape(-1)]))
    want = torch.autograd.grad(moe.grouped_linear(x, w, off), (x, w), dy)
    assert torch.equal(dx, want[0]) and torch.equal(dw, want[1])


@pytest.mark.gpu
def test_group_rows_of_the_largest_batch():
    """2^23 rows over 256 experts, a share of them dropped."""
    R, E = 1 << 23, 256
    g = torch.Generator("cuda").manual_seed(1)
    ids = torch.randint(-1, E + 1, (R // 8, 8), generator=g, device="cuda", dtype=torch.int32)
    off, src, inv = moe.group_rows(ids, E)
    flat = ids.reshape(-1)
    live = (flat >= 0) & (flat < E)
    n = int(live.sum())
    order = torch.argsort(torch.where(live, flat, E), stable=True)[:n]
    assert torch.equal(src[:n].long(), order) and not src[n:].any()
    want = torch.full((R,), -1, dtype=torch.int32, device="cuda")
    want[order] = torch.arange(n, dtype=torch.int32, device="cuda")
    assert torch.equal(inv.reshape(-1), want)
    assert off.tolist() == [0] + torch.bincount(flat[live], minlength=E).cumsum(0).tolist()
