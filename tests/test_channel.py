"""8-bit integers with a scale per token and channel: the quantisers, the dense product
and the "int8" bank bit for bit (integer sums are exact, and what follows them is a
known order of fp32 operations), refusals."""
import ctypes

import numpy as np
import pytest
import torch

import sparse_moe_routed_amd as moe
from oracle import codecs
from oracle import moe as om
from sparse_moe_routed_amd import synth

FAKE = 0x100000  # never dereferenced: the calls below fail validation first

SMALL = synth.Dims(hidden=256, ffn=192, n_experts=32, top_k=4)
WIDE = synth.Dims(hidden=128, ffn=128, n_experts=256, top_k=8)
ODD = synth.Dims(hidden=192, ffn=320, n_experts=16, top_k=2)  # half steps at both ends
FULL = synth.Dims()


def _ld(d):
    return moe.LayerDims(d.hidden, d.ffn, d.n_experts, d.top_k)


# --------------------------------------------------------------------------- CPU
def test_oracle_codec():
    q, s = codecs.int8_row_quantize(np.full((1, 130), 3.5))
    assert (q == 127).all() and s[0] == np.float32(3.5 / 127)
    # rows are apart, zeros are exact, and a code is within half a step of its value
    # (and the fp32 roundings of s and 127 / amax)
    v = codecs.bf16_rne(np.random.default_rng(1).standard_normal((5, 300)))
    v[2, 7], v[3] = 1000.0, 0.0
    q, s = codecs.int8_row_quantize(v)
    assert np.abs(q).max() == 127 and q[2, 7] == 127 and not q[3].any() and s[3] == 0
    d = codecs.int8_row_dequantize(q, s)
    assert (np.abs(d - v) <= 0.5 * s[:, None] + 2.0 ** -22 * np.abs(v)).all()
    # ties to even: 127 / 254 is exact
    q, s = codecs.int8_row_quantize(np.array([[254.0, 1.0, 3.0, -1.0, -3.0, 5.0]]))
    assert q.tolist() == [[127, 0, 2, 0, -2, 2]] and s[0] == 2.0
    q, s = codecs.int8_row_quantize(np.array([[1e-38, 0.0], [np.inf, 1.0], [np.nan, 1.0]]))
    assert not q.any() and s[0] == 0 and np.isnan(s[1:]).all()
    # the bank: a scaled identity is exact
    up = np.stack([np.eye(64) * 2.0, np.eye(64)])
    y = om.forward(np.full((1, 64), 127.0), np.array([[0, 1]]), np.array([[1.0, 0.5]]), om.ExpertBank(up, up, "int8"))
    a = [float(codecs.bf16_rne(np.array([v]))[0]) for v in ((127.0 * 2) ** 2, 127.0 ** 2)]
    assert np.allclose(y, a[0] * 2.0 + 0.5 * a[1], rtol=1e-6)  # s and 1 / s in fp32


def test_validation():
    L = moe.lib()
    for fn in (L.moe_channel_pack, L.moe_channel_quantize):
        args = lambda N=64, K=64, w=FAKE, c=FAKE + (1 << 20), s=FAKE + (2 << 20): (N, K, w, c, s, None)
        for bad in (dict(N=-1), dict(K=0), dict(K=-16), dict(w=None), dict(c=None), dict(s=None),
                    dict(w=FAKE + 8), dict(c=FAKE + 4), dict(s=FAKE + 2), dict(c=FAKE), dict(s=FAKE + 4)):
            assert fn(*args(**bad)) == moe.EINVAL, bad
        assert fn(*args(K=24)) == moe.EUNSUPPORTED
        assert fn(*args(K=(1 << 16) + 16)) == moe.EUNSUPPORTED
    assert L.moe_channel_pack(0, 64, FAKE, FAKE, FAKE, None) == moe.EINVAL
    assert L.moe_channel_pack((1 << 20) + 1, 64, FAKE, FAKE, FAKE, None) == moe.EUNSUPPORTED
    assert L.moe_channel_quantize((1 << 20) + 1, 64, FAKE, FAKE, FAKE, None) == moe.EINVAL
    assert L.moe_channel_quantize(0, 64, None, None, None, None) == moe.OK
    assert L.moe_channel_packed_size(17, 144) == 2 * 2 * 2048 and L.moe_channel_packed_size(0, 64) == 0
    assert L.moe_channel_packed_size(16, 24) == 0 and L.moe_channel_packed_size(16, (1 << 16) + 16) == 0
    pc = L.moe_channel_pack_codes
    for bad in ((0, 64, FAKE, FAKE + 4096), (16, 0, FAKE, FAKE + 4096), (16, 64, None, FAKE), (16, 64, FAKE, None),
                (16, 64, FAKE, FAKE), (16, 64, FAKE + 8, FAKE + 4096), (16, 64, FAKE, FAKE + 4104)):
        assert pc(*bad, None) == moe.EINVAL, bad
    assert pc(16, 40, FAKE, FAKE + 4096, None) == moe.EUNSUPPORTED

    x, c, s, w, ws, y, k = (FAKE + (i << 20) for i in range(7))  # 1 MiB apart

    def mm(M=4, N=64, K=64, c=c, s=s, wc=w, ws=ws, y=y, yd=0):
        return L.moe_channel_matmul(M, N, K, c, s, wc, ws, y, yd, None)

    for bad in (dict(M=-1), dict(N=0), dict(K=0), dict(c=None), dict(s=None), dict(wc=None),
                dict(ws=None), dict(y=None), dict(c=c + 8), dict(wc=w + 1), dict(s=s + 2),
                dict(ws=ws + 1), dict(y=y + 2), dict(yd=2), dict(yd=-1)):
        assert mm(**bad) == moe.EINVAL, bad
    assert mm(K=40) == moe.EUNSUPPORTED and mm(N=(1 << 20) + 1) == moe.EUNSUPPORTED
    assert mm(M=0, c=None, s=None, y=None) == moe.OK and mm(M=0, yd=3) == moe.EINVAL

    need = L.moe_channel_linear_workspace_size(40, 64)
    assert need >= 40 * 64 + 160 and need % 256 == 0
    assert L.moe_channel_linear_workspace_size(-1, 64) == 0 and L.moe_channel_linear_workspace_size(4, 20) == 0

    def lin(M=40, N=64, K=64, x=x, wc=w, s=s, y=y, yd=0, ws=k, nb=need):
        return L.moe_channel_linear(M, N, K, x, wc, s, y, yd, ws, nb, None)

    for bad in (dict(x=None), dict(wc=None), dict(s=None), dict(y=None), dict(x=x + 8), dict(y=y + 4), dict(yd=7)):
        assert lin(**bad) == moe.EINVAL, bad
    for bad in (dict(ws=None), dict(nb=need - 1), dict(ws=k + 16)):
        assert lin(**bad) == moe.EWORKSPACE, bad
    assert lin(M=0, x=None, y=None, ws=None, nb=0) == moe.OK


def test_validation_of_the_bank():
    L = moe.lib()
    d = moe.Dims(2688, 1856, 128, 6)
    sizes = [L.moe_workspace_size(ctypes.byref(d), 4, T) for T in (0, 1, 64, 4096)]
    assert all(s > 0 and s % 256 == 0 for s in sizes) and sizes == sorted(sizes)
    assert sizes[2] <= moe.NOALLOC_SCRATCH_BYTES
    lay = moe.workspace_layout(moe.LayerDims(), "int8", 64)
    assert 0 < lay["act"] < lay["x_q"] < lay["act_q"]

    def fwd(d, ex, nb):
        return L.moe_forward(ctypes.byref(d), 4, FAKE, FAKE, FAKE, ctypes.byref(ex), FAKE, 1, FAKE, nb, None)

    ex = moe.Experts(4, FAKE, FAKE, None, None, FAKE, FAKE)
    assert fwd(d, moe.Experts(4, FAKE, FAKE, None, None, None, None), sizes[2]) == moe.EINVAL  # no scales
    assert fwd(d, ex, 256) == moe.EWORKSPACE
    assert fwd(d, moe.Experts(5, FAKE, FAKE, None, None, FAKE, FAKE), sizes[2]) == moe.EINVAL  # no such format
    # sums past int32 are refused by every call that takes the format
    long = moe.Dims(128, 65600, 16, 2)
    assert L.moe_workspace_size(ctypes.byref(long), 4, 4) == 0 and L.moe_workspace_size(ctypes.byref(long), 3, 4) > 0
    assert L.moe_layer_few_workspace_size(ctypes.byref(long), 4, 4) == 0
    assert fwd(long, ex, 1 << 30) == moe.EUNSUPPORTED
    assert L.moe_quantize_experts(ctypes.byref(long), 4, FAKE, FAKE, FAKE, FAKE, None, None, FAKE, FAKE,
                                  None) == moe.EUNSUPPORTED
    one = moe.Dims(128, 65600, 1, 1)
    assert L.moe_shared_workspace_size(ctypes.byref(one), 4, 4) == 0
    with pytest.raises(moe.MoeError):
        moe.workspace_layout(moe.LayerDims(128, 65600, 16, 2), "int8", 4)
    a = L.moe_quantize_activation
    assert a(4, 4, 60, FAKE, FAKE, None, FAKE, None, 0, None) == moe.EINVAL
    assert a(4, 4, 64, FAKE, None, None, FAKE, None, 0, None) == moe.EINVAL
    assert a(4, 0, 64, FAKE, FAKE, None, FAKE, None, 0, None) == moe.OK


def test_overlapping_buffers_are_refused():
    L = moe.lib()
    M, N, K = 40, 64, 256
    x, c, s, w, ws, y = (FAKE + (i << 20) for i in range(6))  # 1 MiB apart
    wb = L.moe_channel_packed_size(N, K)
    for bad in ((x, x, s), (x, x + 2 * M * K - 16, s), (x, c, x + 4), (x, c, c + M * K - 4)):
        assert L.moe_channel_quantize(M, K, *bad, None) == moe.EINVAL, bad
    for bad in ((x, x + 2 * N * K - 16, s), (x, c, x + 2 * N * K - 4), (x, c, c + wb - 4)):
        assert L.moe_channel_pack(N, K, *bad, None) == moe.EINVAL, bad
    for bad in ((c, c + N * K - 16), (c + wb - 16, c)):
        assert L.moe_channel_pack_codes(N, K, *bad, None) == moe.EINVAL, bad
    for yd, yb in ((0, M * N * 2), (1, M * N * 4)):
        for bad in (c, c + M * K - 16, s, s + M * 4 - 16, w + wb - 16, ws, w - yb + 16):
            assert L.moe_channel_matmul(M, N, K, c, s, w, ws, bad, yd, None) == moe.EINVAL, hex(bad)
    need = L.moe_channel_linear_workspace_size(M, K)
    for m in (M, 4):  # the two kernels, the one
        for bad in (x, x + 2 * m * K - 16, w + wb - 16, s):
            assert L.moe_channel_linear(m, N, K, x, w, s, bad, 0, ws, need, None) == moe.EINVAL, hex(bad)
    assert L.moe_channel_linear(M, N, K, x, w, s, ws + 256, 0, ws, need, None) == moe.EINVAL
    assert L.moe_channel_linear(M, N, K, ws + 256, w, s, y, 0, ws, need, None) == moe.EINVAL


# --------------------------------------------------------------------------- GPU
def _rows(M, K, seed, outliers=True):
    g = torch.Generator().manual_seed(seed)
    x = torch.randn((M, K), generator=g)
    if outliers and M > 2:
        x[::5] *= 100.0
        x[1] = 0.0
        x[2, :K // 2] *= 1e-3
    return x.bfloat16()


def _weight(N, K, seed):
    g = torch.Generator().manual_seed(1000 + seed)
    return (torch.randn((N, K), generator=g) * (0.1 + torch.rand((N, 1), generator=g))).bfloat16()


def _unpack(packed, N, K):
    """Row-major codes [N, K] of packed ones; the padding must be zero."""
    n, kb = (N + 15) // 16, -(-K // 128)
    # [group, step, half, chunk, row, 16] -> [group, row, step, half, chunk, 16]
    full = packed.reshape(n, kb, 2, 4, 16, 16).transpose(0, 4, 1, 2, 3, 5).reshape(n * 16, kb * 128)
    assert not full[N:].any() and not full[:, K:].any()
    return full[:N, :K]


@pytest.mark.gpu
@pytest.mark.parametrize("N,K", [(1, 16), (3, 80), (130, 144), (64, 128), (257, 192), (12, 2688), (9, 4096),
                                 (5, 4112), (3, 65536)])
def test_quantisers_bit_exact(N, K):
    x = _rows(N, K, N + K)
    x[0, 0] = -0.0
    qo, so = codecs.int8_row_quantize(x.float().numpy())
    q, s = moe.channel_quantize(x.cuda())
    assert np.array_equal(q.cpu().numpy(), qo) and np.array_equal(s.cpu().numpy(), so)
    w = moe.channel_pack(x.cuda())
    assert np.array_equal(_unpack(w.codes.cpu().numpy(), N, K), qo) and np.array_equal(w.scales.cpu().numpy(), so)
    again = moe.channel_pack_codes(torch.from_numpy(qo).cuda(), w.scales)
    assert torch.equal(again.codes, w.codes) and again.shape == (N, K)
    q, s = moe.channel_quantize(torch.full((2, K), 1e-38).bfloat16().cuda())
    assert not q.any() and not s.any()
    if K % 64 == 0:
        q2, none, s2 = moe.quantize_activation(x.cuda(), "int8")
        assert none is None and np.array_equal(q2.cpu().numpy(), qo) and np.array_equal(s2.cpu().numpy(), so)


@pytest.mark.gpu
def test_codes_at_the_borders():
    """Every bf16 value next to a border between two codes, for maxima whose 127 / amax
    is exact and for ones where it is rounded either way; huge and small rows."""
    rows = []
    for amax in (254.0, 127.0, 1.0, 3.0, 2.0 ** 100, 2.0 ** -90, 3.3895314e38, 1.1):
        a = torch.tensor(amax).bfloat16()
        grid = ((torch.arange(-254, 255) / 254.0).double() * a.double()).bfloat16()
        bits = grid.view(torch.int16)
        near = torch.cat([grid, (bits + 1).view(torch.bfloat16), (bits - 1).view(torch.bfloat16)])
        near = torch.where(near.float().abs() <= a.float(), near, a)  # a step past the maximum, or off -0
        rows.append(torch.cat([a.view(1), near, torch.zeros(1536 - 1 - near.numel(), dtype=torch.bfloat16)]))
    x = torch.stack(rows)
    q, s = moe.channel_quantize(x.cuda())
    qo, so = codecs.int8_row_quantize(x.float().numpy())
    assert np.array_equal(q.cpu().numpy(), qo) and np.array_equal(s.cpu().numpy(), so)


def _value(qa, sa, qw, sw):
    """fp32 results as the header defines them: the exact sum's fp32 value times the
    row's scale, then times the channel's."""
    acc = qa.astype(np.float64) @ qw.astype(np.float64).T  # below 2^53: exact
    return acc.astype(np.float32) * sa[:, None] * sw[None, :]


def _same(got, want):
    return np.array_equal(got.float().cpu().numpy(), want, equal_nan=True)


SHAPES = [(1, 1, 16), (1, 3712, 2688), (3, 37, 64), (7, 130, 144), (16, 64, 128), (17, 33, 1856),
          (32, 200, 400), (33, 64, 2688), (77, 301, 336), (128, 129, 256), (129, 130, 144), (200, 1, 128),
          (300, 515, 1856), (513, 768, 208), (2900, 3000, 80), (4096, 1856, 320), (150, 1000, 2688),
          (500, 3700, 2000), (1000, 3700, 1840), (1500, 9000, 400), (2, 40, 8192), (40, 40, 8192), (40, 8200, 144),
          (100, 8200, 144), (1100, 4400, 80), (1100, 2300, 80), (600, 2300, 96)]


@pytest.mark.gpu
@pytest.mark.parametrize("M,N,K", SHAPES)
def test_matmul(M, N, K):
    x, w = _rows(M, K, M + N + K), _weight(N, K, M + N)
    W = moe.channel_pack(w.cuda())
    q, s = moe.channel_quantize(x.cuda())
    want = _value(*codecs.int8_row_quantize(x.float().numpy()), *codecs.int8_row_quantize(w.float().numpy()))
    for dt in (torch.bfloat16, torch.float32):
        store = torch.full((M * N + 640,), 7.0, dtype=dt, device="cuda")
        y = moe.channel_matmul(q, s, W, y=store[:M * N].view(M, N))
        assert _same(y, torch.from_numpy(want).to(dt).float().numpy())
        assert (store[M * N:] == 7.0).all()
        z = moe.channel_linear(x.cuda(), W, y_dtype=dt)
        assert torch.equal(y, z)
    assert moe.channel_linear(x.cuda(), W).dtype == torch.bfloat16


@pytest.mark.gpu
@pytest.mark.parametrize("M", [1, 16, 40, 150, 700])
def test_largest_sums(M):
    """Codes of -128 and 127 over the longest K: sums of 2^30 either way."""
    K, N = 65536, 48
    rng = np.random.default_rng(M)
    qa = rng.choice(np.array([-128, 127], np.int8), (M, 1)).repeat(K, 1)
    qw = rng.choice(np.array([-128, 127], np.int8), (N, 1)).repeat(K, 1)
    qw[5] = rng.integers(-128, 128, K)
    sa, sw = np.full(M, 2.0 ** -20, np.float32), np.full(N, 0.75, np.float32)
    W = moe.channel_pack_codes(torch.from_numpy(qw).cuda(), torch.from_numpy(sw).cuda())
    y = moe.channel_matmul(torch.from_numpy(qa).cuda(), torch.from_numpy(sa).cuda(), W, y_dtype=torch.float32)
    assert _same(y, _value(qa, sa, qw, sw))


@pytest.mark.gpu
@pytest.mark.parametrize("M,N", [(70000, 24), (3, 70000), (150, 70000), (70000, 32768)])
def test_past_32_bits(M, N):
    """Codes, weights or results of more than 4 GB: the last rows and channels."""
    K = 65536 if min(M, N) < 1000 else 64
    x = torch.empty((M, K), dtype=torch.bfloat16, device="cuda").normal_()
    w = torch.empty((N, K), dtype=torch.bfloat16, device="cuda").normal_()
    W = moe.channel_pack(w)
    y = moe.channel_linear(x, W)
    q, s = moe.channel_quantize(x)
    xs, ws = x[-20:].float().cpu().numpy(), w[-40:].float().cpu().numpy()
    want = _value(*codecs.int8_row_quantize(xs), *codecs.int8_row_quantize(ws))
    for got in (y, moe.channel_matmul(q, s, W)):
        assert _same(got[-20:, -40:], torch.from_numpy(want).bfloat16().float().numpy())


@pytest.mark.gpu
@pytest.mark.parametrize("M", [5, 20, 40, 300])
def test_rows_and_channels_are_apart(M):
    """NaN and infinities: their row of y, or their column, is NaN; no other changes."""
    x, w = _rows(M, 144, M), _weight(130, 144, M)
    want = moe.channel_linear(x.cuda(), moe.channel_pack(w.cuda()))
    x2, w2 = x.clone(), w.clone()
    x2[3], x2[4, 140] = float("nan"), float("-inf")
    w2[5, 7], w2[129, 143] = float("nan"), float("inf")
    got = moe.channel_linear(x2.cuda(), moe.channel_pack(w2.cuda()))
    rows, cols = [i for i in range(M) if i not in (3, 4)], [n for n in range(130) if n not in (5, 129)]
    assert torch.equal(got[rows][:, cols], want[rows][:, cols])
    assert got[[3, 4]].isnan().all() and got[:, [5, 129]].isnan().all()
    # a zero sum stays zero where the scales' product is past fp32's range
    big = torch.zeros((M, 16))
    big[:, 0], big[1, 1] = 3e38, 3e38
    v = torch.zeros((3, 16))
    v[0, 1], v[1, 0], v[2, 2] = 3e38, 3e38, 1.0
    y = moe.channel_linear(big.bfloat16().cuda(), moe.channel_pack(v.bfloat16().cuda()))
    assert not y[0, 0].any() and not y[:, 2].any() and y[:, 1].isinf().all() and y[1, 0].isinf()


@pytest.mark.gpu
def test_refusals_of_the_binding():
    x = _rows(4, 64, 1).cuda()
    W = moe.channel_pack(_weight(32, 64, 1).cuda())
    q, s = moe.channel_quantize(x)
    e = lambda *shape, dtype=torch.bfloat16: torch.empty(shape, dtype=dtype, device="cuda")
    for bad in (lambda: moe.channel_linear(x.float(), W), lambda: moe.channel_linear(x.cpu(), W),
                lambda: moe.channel_linear(x[:, :32], W), lambda: moe.channel_linear(x[0], W),
                lambda: moe.channel_linear(x, W, y=e(4, 31)), lambda: moe.channel_linear(x, W, y=e(4, 32).cpu()),
                lambda: moe.channel_linear(x, W, y=e(4, 32, dtype=torch.float16)),
                lambda: moe.channel_linear(x, W, y=e(4, 32), y_dtype=torch.float32),
                lambda: moe.channel_linear(x, W, y_dtype=torch.float16),
                lambda: moe.channel_linear(x, W, ws=torch.empty(9, device="cuda")),
                lambda: moe.channel_linear(x, moe.ChannelWeight(W.codes, W.scales[:8], W.shape)),
                lambda: moe.channel_linear(x, moe.ChannelWeight(W.codes[16:], W.scales, W.shape)),
                lambda: moe.channel_linear(x, moe.ChannelWeight(W.codes, W.scales, (32, 128))),
                lambda: moe.channel_pack_codes(q.float(), s), lambda: moe.channel_pack_codes(q, s[:2]),
                lambda: moe.channel_matmul(q, s[:2], W), lambda: moe.channel_matmul(q.t(), s, W),
                lambda: moe.channel_matmul(q.view(torch.uint8), s, W),
                lambda: moe.channel_pack(x.float()), lambda: moe.channel_quantize(x.t()),
                lambda: moe.channel_packed_size(4, 65552)):
        with pytest.raises(ValueError):
            bad()
    with pytest.raises(moe.MoeError) as err:
        moe.channel_quantize(e(4, 24))
    assert err.value.status == moe.EUNSUPPORTED
    with pytest.raises(moe.MoeError) as err:
        moe.channel_linear(x.repeat(10, 1), W, ws=torch.empty(256, dtype=torch.uint8, device="cuda"))
    assert err.value.status == moe.EWORKSPACE
    assert moe.channel_linear(x[:0], W).shape == (0, 32)


@pytest.mark.gpu
@pytest.mark.parametrize("M", [1, 32, 33, 200])
def test_linear_captured_and_on_another_stream(M):
    x, w = _rows(M, 400, M).cuda(), _weight(200, 400, M)
    W = moe.channel_pack(w.cuda())
    ws = moe.channel_linear_workspace(M, 400)
    y = moe.channel_linear(x, W, ws=ws)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        moe.channel_linear(x, W, y=y, ws=ws)
    for k in range(4):
        x.copy_(_rows(M, 400, 100 + k))
        want = moe.channel_linear(x, W)
        y.fill_(float("nan"))
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(y, want)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        z = moe.channel_linear(x, W)
    side.synchronize()
    assert torch.equal(z, want)


# ---- the bank
_layers = {}


class Layer:
    def __init__(self, dims):
        self.dims, self.ld = dims, _ld(dims)
        self.w_r, self.b = synth.make_router(0, dims)
        self.up, self.down = synth.make_experts(0, dims)
        self.router = moe.pack_router(self.w_r.cuda(), self.b.cuda(), self.ld)
        self.bank = moe.quantize_experts(self.up.cuda(), self.down.cuda(), "int8", self.ld)


def layer(dims):
    if dims not in _layers:
        _layers[dims] = Layer(dims)
    return _layers[dims]


@pytest.mark.gpu
def test_bank_codes_bit_exact():
    L = layer(ODD)
    for e in (0, 15):
        for src, q, s in ((L.up, L.bank.up, L.bank.up_s), (L.down, L.bank.down, L.bank.down_s)):
            qo, so = codecs.int8_row_quantize(src[e].float().numpy())
            assert np.array_equal(_unpack(q[e].cpu().numpy(), *src[e].shape), qo)
            assert np.array_equal(s[e].cpu().numpy(), so)


def _forward(L, x, ids, gates):
    """The layer bit for bit: (y fp32 [T, H], a of each flat entry)."""
    qx, sx = codecs.int8_row_quantize(x.float().numpy())
    T, k = ids.shape
    flat = ids.reshape(-1)
    a = np.zeros((T * k, L.dims.ffn))
    o = np.zeros((T * k, L.dims.hidden), np.float32)
    for e in np.unique(flat):
        r = np.nonzero(flat == e)[0]
        h = _value(qx[r // k], sx[r // k], *codecs.int8_row_quantize(L.up[int(e)].float().numpy()))
        a[r] = codecs.bf16_rne(np.maximum(h, 0).astype(np.float64) ** 2)
    qa, sa = codecs.int8_row_quantize(a)
    for e in np.unique(flat):
        r = np.nonzero(flat == e)[0]
        v = _value(qa[r], sa[r], *codecs.int8_row_quantize(L.down[int(e)].float().numpy()))
        o[r] = v * gates.reshape(-1)[r, None]
    y = np.zeros((T, L.dims.hidden), np.float32)
    for j in range(k):
        y = y + o.reshape(T, k, -1)[:, j]
    return y, a, qa, sa


@pytest.mark.gpu
@pytest.mark.parametrize("name,T", [("ODD", 1), ("ODD", 5), ("ODD", 127), ("ODD", 128), ("ODD", 300), ("SMALL", 64),
                                    ("SMALL", 255), ("SMALL", 256), ("SMALL", 700), ("WIDE", 3), ("WIDE", 600),
                                    ("FULL", 2)])
def test_forward_bit_exact(name, T):
    L = layer(globals()[name])
    x = synth.make_tokens(T, L.dims, outliers=True)
    ids, gates = moe.route(x.cuda(), L.router, L.ld)
    ws = moe.workspace(L.ld, "int8", T)
    y = moe.forward(x.cuda(), ids, gates, L.bank, L.ld, ws=ws)
    want, a, qa, sa = _forward(L, x, ids.cpu().numpy(), gates.cpu().numpy())
    lay, R, F = moe.workspace_layout(L.ld, "int8", T), T * L.dims.top_k, L.dims.ffn
    order = ws[lay["sorted_src"]:lay["sorted_src"] + R * 4].view(torch.int32).cpu().numpy()
    act = ws[lay["act"]:lay["act"] + R * F * 2].view(torch.bfloat16).view(R, F)
    assert np.array_equal(act.double().cpu().numpy(), a[order])
    codes = ws[lay["act_q"]:lay["act_q"] + R * F].view(torch.int8).view(R, F).cpu().numpy()
    at = lay["act_q"] + -(-R * F // 256) * 256
    scales = ws[at:at + R * 4].view(torch.float32).cpu().numpy()
    assert np.array_equal(codes, qa[order]) and np.array_equal(scales, sa[order])
    assert np.array_equal(y.cpu().numpy(), want)
    # the oracle's float64 result: the same codes but where a value of the
    # intermediate lies next to a border, so equal in the mean
    ref = om.forward(x.float().numpy(), ids.cpu().numpy(), gates.double().cpu().numpy(),
                     om.ExpertBank(L.up, L.down, "int8"))
    assert np.linalg.norm(want - ref) <= 1e-3 * np.linalg.norm(ref)
    yb = moe.forward(x.cuda(), ids, gates, L.bank, L.ld, y_dtype=torch.bfloat16, ws=ws)
    assert torch.equal(yb, y.bfloat16())


@pytest.mark.gpu
@pytest.mark.parametrize("name,T", [("FULL", 4096), ("FULL", 700), ("ODD", 2000), ("WIDE", 1111)])
def test_long_batch_is_its_parts(name, T):
    """A token's result does not depend on the batch: the long batches' tiles against
    the short ones', bit for bit, and the same every time."""
    L = layer(globals()[name])
    x = synth.make_tokens(T, L.dims, outliers=True).cuda()
    ids, gates = moe.route(x, L.router, L.ld)
    y = moe.forward(x, ids, gates, L.bank, L.ld)
    parts = [moe.forward(x[i:i + 100], ids[i:i + 100], gates[i:i + 100], L.bank, L.ld) for i in range(0, T, 100)]
    assert torch.equal(y, torch.cat(parts))
    ws = moe.workspace(L.ld, "int8", T)
    for _ in range(4):
        ws.fill_(255)  # NaN in every float format: what no kernel has written shows
        assert torch.equal(moe.forward(x, ids, gates, L.bank, L.ld, ws=ws), y)


@pytest.mark.gpu
def test_other_calls_with_the_bank():
    L = layer(SMALL)
    x = synth.make_tokens(9, SMALL).cuda()
    ids, gates = moe.route(x, L.router, L.ld)
    want = moe.forward(x, ids, gates, L.bank, L.ld)
    assert torch.equal(moe.forward_noalloc(x, ids, gates, L.bank, L.ld), want)
    cache = moe.ExpertCache(L.bank, 32, L.ld)
    for _ in range(2):
        y, st = moe.forward_cached(x, ids, gates, cache, L.ld)
        assert torch.equal(y, want)
    assert st["misses"] == 0 and st["hits"] == len(torch.unique(ids))
    y, st = moe.forward_cached(x, ids, gates, moe.ExpertCache(L.bank, 31, L.ld), L.ld)
    assert torch.equal(y, want) and st["bytes_uploaded"] == st["misses"] * (192 * 256 + 256 * 256)
    evs = [torch.cuda.Event(enable_timing=True) for _ in range(moe.N_TIMED_EVENTS)]
    for e in evs:
        e.record()
    y = moe.forward_timed(x, ids, gates, L.bank, [e.cuda_event for e in evs], L.ld)
    torch.cuda.synchronize()
    assert torch.equal(y, want) and evs[0].elapsed_time(evs[6]) > 0
    # dropped slots contribute nothing; no tokens are a no-op
    bad, g2 = ids.clone(), gates.clone()
    bad[:, 1] = 99
    y = moe.forward(x, bad, g2, L.bank, L.ld)
    g2[:, 1] = 0
    assert torch.equal(y, moe.forward(x, ids, g2, L.bank, L.ld))
    bad[:] = -1
    assert not moe.forward(x, bad, gates, L.bank, L.ld).any()
    assert moe.forward(x[:0], ids[:0], gates[:0], L.bank, L.ld).shape == (0, 256)
    # a few tokens: as route and forward
    y, i2, g2 = moe.layer_few(x, L.router, L.bank, L.ld)
    assert torch.equal(y, want) and torch.equal(i2, ids) and torch.equal(g2, gates)
    with pytest.raises(ValueError):
        moe.forward(x, ids, gates, moe.ExpertBank("int8", L.bank.up, L.bank.down, None, None, L.bank.up_s,
                                                  L.bank.down_s[:16]), L.ld)


@pytest.mark.gpu
@pytest.mark.parametrize("T", [1, 40, 300])
def test_shared_expert(T):
    """Every token at one expert with weight 1: two dense products with the square
    between them, bit for bit."""
    sd = moe.shared_dims(256, 448)
    up, down = synth.make_shared_expert(0, 256, 448)
    bank = moe.quantize_experts(up[None].cuda(), down[None].cuda(), "int8", sd)
    x = synth.make_tokens(T, SMALL).cuda()
    y = moe.shared_forward(x, bank, sd)
    h = moe.channel_linear(x, moe.channel_pack(up.cuda()), y_dtype=torch.float32)
    a = h.clamp(min=0).double().square().cpu().numpy()
    a = torch.from_numpy(codecs.bf16_rne(a)).bfloat16().cuda()
    assert torch.equal(y, moe.channel_linear(a, moe.channel_pack(down.cuda()), y_dtype=torch.float32))
    z = torch.ones_like(y)
    moe.shared_forward(x, bank, sd, y=z, accumulate=True)
    assert torch.equal(z, y + 1.0)


@pytest.mark.gpu
@pytest.mark.parametrize("T", [9, 300])
def test_tokens_of_nan_leave_the_others_in_the_experts(T):
    L = layer(SMALL)
    x = synth.make_tokens(T, SMALL).cuda()
    ids, gates = moe.route(x, L.router, L.ld)
    want = moe.forward(x, ids, gates, L.bank, L.ld)
    x[3, 7], x[4, 200], x[5] = float("nan"), float("inf"), float("-inf")
    y = moe.forward(x, ids, gates, L.bank, L.ld)
    keep = [t for t in range(T) if t not in (3, 4, 5)]
    assert torch.equal(y[keep], want[keep]) and not y[3:6].any()


@pytest.mark.gpu
@pytest.mark.parametrize("T", [1, 9, 300])
def test_block_captured_and_on_two_streams(T):
    """A decoder block in 8-bit integers, pre-norm, routed and shared experts and a
    projection, captured and replayed with new tokens and routing; two at once on two
    streams, each with its own workspace."""
    L = layer(ODD)
    sd, d = moe.shared_dims(192, 320), L.dims
    shared = moe.quantize_experts(L.up[:1].cuda(), L.down[:1].cuda(), "int8", sd)
    W = moe.channel_pack(_weight(192, 192, 4).cuda())
    x = synth.make_tokens(T, d).cuda()

    def space():
        return (moe.workspace(L.ld, "int8", T), moe.shared_workspace(sd, "int8", T),
                moe.channel_linear_workspace(T, 192), moe.route_workspace(L.ld, T))

    def step(x, y, p, ws):
        h = moe.prenorm(x)
        ids, gates = moe.route(h, L.router, L.ld, ws=ws[3])
        moe.forward(h, ids, gates, L.bank, L.ld, y=y, ws=ws[0])
        moe.shared_forward(h, shared, sd, y=y, accumulate=True, ws=ws[1])
        return moe.channel_linear(y.bfloat16(), W, y=p, ws=ws[2])

    def outs():
        return torch.empty((T, 192), device="cuda"), torch.empty((T, 192), dtype=torch.bfloat16, device="cuda")

    ws, (y, p) = space(), outs()
    step(x, y, p, ws)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        step(x, y, p, ws)
    for k in range(4):
        x.copy_(torch.roll(synth.make_tokens(T + 7 * k, d, outliers=k % 2 == 1)[:T], k, 1))
        want = step(x, *outs(), space()).clone()
        p.fill_(float("nan"))
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(p, want)
    streams = [torch.cuda.Stream() for _ in range(2)]
    both = [(outs(), space()) for _ in streams]
    torch.cuda.synchronize()
    for _ in range(10):
        for s, ((y, p), w) in zip(streams, both):
            with torch.cuda.stream(s):
                step(x, y, p, w)
    torch.cuda.synchronize()
    assert torch.equal(both[0][0][1], want) and torch.equal(both[1][0][1], want)


# (M, N, K) whose rows of y are no multiple of 16 bytes, in each of the larger tiles:
# 256 x 256, 128 x 256, 128 x 128 and 64 x 128
ODD_ROWS = [(2900, 3001, 80), (2900, 3002, 80), (2900, 3004, 80), (1100, 4399, 80), (1100, 4402, 80), (1100, 2301, 80),
            (1100, 2302, 80), (1100, 2300, 80), (600, 2301, 96), (600, 2302, 96)]


@pytest.mark.gpu
@pytest.mark.parametrize("M,N,K", ODD_ROWS)
def test_odd_rows_of_large_tiles(M, N, K):
    x, w = _rows(M, K, M + N + K), _weight(N, K, M + N)
    W = moe.channel_pack(w.cuda())
    q, s = moe.channel_quantize(x.cuda())
    want = _value(*codecs.int8_row_quantize(x.float().numpy()), *codecs.int8_row_quantize(w.float().numpy()))
    for dt in (torch.bfloat16, torch.float32):
        store = torch.full((M * N + 1280,), 7.0, dtype=dt, device="cuda")
        y = moe.channel_matmul(q, s, W, y=store[640:640 + M * N].view(M, N))
        assert _same(y, torch.from_numpy(want).to(dt).float().numpy())
        assert (store[:640] == 7.0).all() and (store[640 + M * N:] == 7.0).all()
