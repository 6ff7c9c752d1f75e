"""moe_layer_few: router and experts of at most 16 tokens in two kernels, against
the float64 oracle and against moe_route + moe_forward; its refusals, streams
and graphs."""
import ctypes

import numpy as np
import pytest
import torch

import sparse_moe_routed_amd as moe
from oracle import moe as om
from sparse_moe_routed_amd import synth

FAKE = 0x100000  # never dereferenced: the calls below fail validation first

# max |delta| over rms of the oracle output, the layer's own gates: the widest
# step is a code of the intermediate that lies within fp32 rounding of a border
# and falls on the other side (BF16 2^-8, E4M3 2^-3, E2M1 2^-1 of one of
# top_k * F terms)
TOL = {"bf16": 2e-2, "fp8": 5e-2, "nvfp4": 1e-1}
FULL = synth.Dims()
SMALL = synth.Dims(hidden=256, ffn=192, n_experts=32, top_k=4)
WIDE = synth.Dims(hidden=128, ffn=128, n_experts=256, top_k=8)
ODD = synth.Dims(hidden=192, ffn=320, n_experts=16, top_k=2)   # half-empty last units
ONE = synth.Dims(hidden=64, ffn=64, n_experts=16, top_k=1)     # smallest
LONG = synth.Dims(hidden=64, ffn=3712, n_experts=16, top_k=3)  # one expert's rows fill the stage


def _ld(d):
    return moe.LayerDims(d.hidden, d.ffn, d.n_experts, d.top_k)


# --------------------------------------------------------------------------- CPU
def test_workspace_size():
    d = moe.Dims(2688, 1856, 128, 6)
    f = moe.lib().moe_layer_few_workspace_size
    last = 0
    for T in range(17):
        n = f(ctypes.byref(d), 0, T)
        assert n % 256 == 0 and n >= last and n >= T * 6 * 1856 * 2
        last = n
    assert f(ctypes.byref(d), 0, 17) == 0 and f(ctypes.byref(d), 0, -1) == 0
    assert f(ctypes.byref(d), 9, 4) == 0 and f(None, 0, 4) == 0
    assert f(ctypes.byref(moe.Dims(2690, 1856, 128, 6)), 0, 4) == 0


def test_validation():
    d = moe.Dims(2688, 1856, 128, 6)
    ex = moe.Experts(0, FAKE, FAKE, None, None, None, None)
    r = moe.Router(FAKE, None)
    need = moe.lib().moe_layer_few_workspace_size(ctypes.byref(d), 0, 4)

    def call(dims=d, T=4, x=FAKE, router=r, e=ex, ids=FAKE, gates=FAKE, y=FAKE, yd=1, ws=FAKE, wsb=need):
        return moe.lib().moe_layer_few(
            dims if dims is None else ctypes.byref(dims), T, x,
            router if router is None else ctypes.byref(router), e if e is None else ctypes.byref(e),
            ids, gates, y, yd, ws, wsb, None)

    for bad in (dict(dims=None), dict(T=-1), dict(x=None), dict(router=None), dict(e=None),
                dict(router=moe.Router(None, None)), dict(ids=None), dict(gates=None), dict(y=None),
                dict(yd=2), dict(dims=moe.Dims(2688, 1856, 128, 129)),
                dict(e=moe.Experts(9, FAKE, FAKE, None, None, None, None)),
                dict(e=moe.Experts(0, None, FAKE, None, None, None, None)),
                dict(e=moe.Experts(1, FAKE, FAKE, None, None, None, None)),
                dict(e=moe.Experts(2, FAKE, FAKE, None, None, FAKE, FAKE)),
                dict(x=FAKE + 8), dict(y=FAKE + 8), dict(ids=FAKE + 2), dict(gates=FAKE + 1),
                dict(router=moe.Router(FAKE + 2, None)), dict(router=moe.Router(FAKE, FAKE + 2)),
                dict(e=moe.Experts(0, FAKE + 8, FAKE, None, None, None, None))):
        assert call(**bad) == moe.EINVAL, bad
    for bad in (dict(T=17), dict(dims=moe.Dims(2688, 1856, 128, 9)), dict(dims=moe.Dims(2690, 1856, 128, 6))):
        assert call(**bad) == moe.EUNSUPPORTED, bad
    # as two calls: the workspaces of both
    for fmt, T, dims in ((3, 4, d), (0, 16, d), (2, 8, d), (1, 16, moe.Dims(64, 3776, 16, 1))):
        n = moe.lib().moe_layer_few_workspace_size(ctypes.byref(dims), fmt, T)
        assert n >= (moe.lib().moe_route_workspace_size(ctypes.byref(dims), T) +
                     moe.lib().moe_workspace_size(ctypes.byref(dims), fmt, T))
        e = moe.Experts(fmt, FAKE, FAKE, FAKE, FAKE, FAKE, FAKE)
        assert call(dims=dims, T=T, e=e, wsb=n - 1) == moe.EWORKSPACE
    for bad in (dict(ws=None), dict(wsb=need - 1), dict(ws=FAKE + 16)):
        assert call(**bad) == moe.EWORKSPACE, bad
    assert call(T=0, x=None, router=None, ids=None, gates=None, y=None, ws=None, wsb=0) == moe.OK


# --------------------------------------------------------------------------- GPU
class Layer:
    def __init__(self, dims, seed=0):
        self.dims, self.ld = dims, _ld(dims)
        self.w_r, self.b = synth.make_router(seed, dims)
        self.up, self.down = synth.make_experts(seed, dims)
        self.router = moe.pack_router(self.w_r.cuda(), self.b.cuda(), self.ld)
        self.up_d, self.down_d = self.up.cuda(), self.down.cuda()
        self.banks = {}

    def bank(self, fmt):
        if fmt not in self.banks:
            self.banks[fmt] = moe.quantize_experts(self.up_d, self.down_d, fmt, self.ld)
        return self.banks[fmt]


_layers = {}


def layer(dims):
    if dims not in _layers:
        _layers[dims] = Layer(dims)
    return _layers[dims]


def check(L, fmt, x, y_dtype=torch.float32):
    """Against the oracle: the same experts (none of these seeds has a near-tie),
    gates within fp32 rounding of 6 logits and their softmax, y within TOL."""
    y, ids, gates = moe.layer_few(x.cuda(), L.router, L.bank(fmt), L.ld, y_dtype=y_dtype)
    ids_o, g_o, gap, _ = om.route(x.float().numpy(), L.w_r.numpy(), L.b.numpy(), L.dims.top_k)
    assert gap.min() > om.NEAR_TIE
    assert np.array_equal(ids.cpu().numpy(), ids_o)
    assert np.abs(gates.cpu().numpy() - g_o).max() <= 2e-6
    bank = om.ExpertBank(L.up, L.down, fmt).preload(np.unique(ids_o), threads=8)
    ref = om.forward(x.float().numpy(), ids_o, g_o, bank)
    rms = np.sqrt(np.mean(ref ** 2))
    err = np.abs(y.double().cpu().numpy() - ref).max() / rms
    step = 0.0 if y_dtype == torch.float32 else 2.0 ** -8 * np.abs(ref).max() / rms
    print(f"T={x.shape[0]} {fmt}: max|d|/rms {err:.2e}", flush=True)
    assert err <= TOL[fmt] + step
    # the two calls on the same batch: other summation order only
    i2, g2 = moe.route(x.cuda(), L.router, L.ld)
    assert torch.equal(ids, i2) and (gates - g2).abs().max() <= 2e-6
    y2 = moe.forward(x.cuda(), i2, g2, L.bank(fmt), L.ld)
    assert (y.float() - y2).abs().max().item() / rms <= TOL[fmt] + step
    return y, ids, gates


@pytest.mark.gpu
@pytest.mark.parametrize("fmt", ["bf16", "fp8", "nvfp4"])
@pytest.mark.parametrize("name,T", [("ONE", 1), ("ONE", 16), ("ODD", 1), ("ODD", 3), ("ODD", 16),
                                    ("SMALL", 2), ("SMALL", 13), ("WIDE", 1), ("WIDE", 16),
                                    ("LONG", 16), ("LONG", 5)])
def test_matches_oracle(name, T, fmt):
    L = layer(globals()[name])
    check(L, fmt, synth.make_tokens(T, L.dims))


@pytest.mark.gpu
@pytest.mark.parametrize("fmt,T", [("bf16", 1), ("bf16", 7), ("fp8", 4), ("nvfp4", 1), ("fp8", 16),
                                   ("nvfp4", 16)])
def test_full_width(fmt, T):
    L = layer(FULL)
    check(L, fmt, synth.make_tokens(T, FULL), torch.bfloat16 if T == 7 else torch.float32)


@pytest.mark.gpu
@pytest.mark.parametrize("fmt", ["bf16", "fp8", "nvfp4"])
def test_every_token_on_the_same_experts(fmt):
    L = layer(SMALL)
    x = synth.make_tokens(1, SMALL).repeat(16, 1)
    y, ids, gates = check(L, fmt, x)
    assert (ids == ids[0]).all() and (y == y[0]).all()


@pytest.mark.gpu
def test_zero_tokens_and_zero_rows():
    L = layer(SMALL)
    y, ids, gates = moe.layer_few(torch.empty((0, 256), dtype=torch.bfloat16, device="cuda"), L.router,
                                  L.bank("bf16"), L.ld)
    assert y.shape == (0, 256) and ids.shape == (0, 4)
    x = torch.zeros((3, 256), dtype=torch.bfloat16, device="cuda")
    for fmt in ("bf16", "fp8", "nvfp4"):
        y, ids, gates = moe.layer_few(x, L.router, L.bank(fmt), L.ld)
        assert not y.any()
        i2, g2 = moe.route(x, L.router, L.ld)
        assert torch.equal(ids, i2)
    # no bias, all logits equal: ties go to the lowest expert
    r = moe.PackedRouter(torch.zeros_like(L.router.w_packed), None)
    y, ids, gates = moe.layer_few(x, r, L.bank("bf16"), L.ld)
    assert (ids.cpu() == torch.arange(4)).all() and (gates == 0.25).all()


@pytest.mark.gpu
def test_a_token_of_nan_leaves_the_others():
    L = layer(SMALL)
    x = synth.make_tokens(5, SMALL).cuda()
    want, ids, _ = moe.layer_few(x, L.router, L.bank("bf16"), L.ld)
    x2 = x.clone()
    x2[3, 7] = float("nan")
    y, i2, _ = moe.layer_few(x2, L.router, L.bank("bf16"), L.ld)
    for t in (0, 1, 2, 4):
        assert torch.equal(i2[t], ids[t])
        assert (y[t] - want[t]).abs().max() <= 1e-5 * want[t].abs().max()


@pytest.mark.gpu
@pytest.mark.parametrize("fmt", ["bf16", "nvfp4"])
def test_repeats_bit_for_bit_and_writes_only_its_outputs(fmt):
    L = layer(SMALL)
    T = 6
    x = synth.make_tokens(T, SMALL).cuda()
    need = moe.layer_few_workspace(L.ld, fmt, T).numel()
    ws = torch.full((need + 4096,), 0xA5, dtype=torch.uint8, device="cuda")
    y = torch.full((T + 3, 256), 7.0, device="cuda")
    ids = torch.full((T + 3, 4), -9, dtype=torch.int32, device="cuda")
    gates = torch.full((T + 3, 4), 7.0, device="cuda")
    first = None
    for _ in range(5):
        moe.layer_few(x, L.router, L.bank(fmt), L.ld, y=y[:T], ids=ids[:T], gates=gates[:T],
                      ws=ws[:need])
        got = (y.clone(), ids.clone(), gates.clone())
        if first is not None:
            assert all(torch.equal(a, b) for a, b in zip(first, got))
        first = got
    assert (y[T:] == 7.0).all() and (ids[T:] == -9).all() and (gates[T:] == 7.0).all()
    assert (ws[need:] == 0xA5).all()


@pytest.mark.gpu
def test_two_streams_and_graph_replay():
    L = layer(FULL)
    xs = [synth.make_tokens(T, FULL).cuda() for T in (3, 5)]
    bank = L.bank("nvfp4")
    want = [moe.layer_few(x, L.router, bank, L.ld)[0].clone() for x in xs]
    streams = [torch.cuda.Stream() for _ in xs]
    ws = [moe.layer_few_workspace(L.ld, "nvfp4") for _ in xs]
    out = [torch.empty_like(w) for w in want]
    torch.cuda.synchronize()
    for _ in range(8):
        for s, x, o, w in zip(streams, xs, out, ws):
            with torch.cuda.stream(s):
                moe.layer_few(x, L.router, bank, L.ld, y=o, ws=w)
    torch.cuda.synchronize()
    assert all(torch.equal(o, w) for o, w in zip(out, want))
    x, y, ids, gates = xs[0], out[0], torch.empty((3, 6), dtype=torch.int32, device="cuda"), torch.empty((3, 6), device="cuda")
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        moe.layer_few(x, L.router, bank, L.ld, y=y, ids=ids, gates=gates, ws=ws[0])
    for k in range(3):
        x.copy_(synth.make_tokens(3 + 10 * k, FULL)[:3])
        ref = [t.clone() for t in moe.layer_few(x, L.router, bank, L.ld)]
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(y, ref[0]) and torch.equal(ids, ref[1]) and torch.equal(gates, ref[2])


@pytest.mark.gpu
def test_refusals_of_the_binding():
    L = layer(SMALL)
    x = synth.make_tokens(4, SMALL).cuda()
    b = L.bank("bf16")
    for a in (x.float(), x[:, :128], x.cpu(), x.t()):
        with pytest.raises(ValueError):
            moe.layer_few(a, L.router, b, L.ld)
    for kw in (dict(y=torch.empty((3, 256), device="cuda")), dict(ids=torch.empty((4, 4), device="cuda")),
               dict(gates=torch.empty((4, 3), device="cuda")), dict(ws=torch.empty(64, device="cuda"))):
        with pytest.raises(ValueError):
            moe.layer_few(x, L.router, b, L.ld, **kw)
    with pytest.raises(moe.MoeError) as e:
        moe.layer_few(synth.make_tokens(17, SMALL).cuda(), L.router, b, L.ld)
    assert e.value.status == moe.EUNSUPPORTED
    with pytest.raises(moe.MoeError) as e:
        moe.layer_few(x, L.router, b, L.ld, ws=torch.empty(256, dtype=torch.uint8, device="cuda"))
    assert e.value.status == moe.EWORKSPACE


@pytest.mark.gpu
def test_decode_step_between_norms():
    """residual_norm, layer_few, residual_norm, as a decoder's stack runs them,
    against the oracle block by block (teacher-forced on the stored x)."""
    L = layer(SMALL)
    x = synth.make_tokens(3, SMALL).cuda()
    w = [torch.rand(256, device="cuda") + 0.5 for _ in range(2)]
    _, h = moe.residual_norm(x, None, pre_weight=w[0])
    for _ in range(3):
        x0, h0 = x.clone(), h.clone()
        y, ids, gates = moe.layer_few(h, L.router, L.bank("bf16"), L.ld)
        x, h = moe.residual_norm(x, y, post_weight=w[1], pre_weight=w[0], scale=0.5)
        hn = h0.float().cpu().numpy()
        ids_o, g_o, gap, _ = om.route(hn, L.w_r.numpy(), L.b.numpy(), 4)
        if gap.min() > om.NEAR_TIE:
            assert np.array_equal(ids.cpu().numpy(), ids_o)
        ref = om.forward(hn, ids.cpu().numpy(), gates.double().cpu().numpy(), om.ExpertBank(L.up, L.down, "bf16"))
        rms = np.sqrt(np.mean(ref ** 2))
        assert np.abs(y.double().cpu().numpy() - ref).max() <= TOL["bf16"] * rms
        xr, _ = om.residual_norm(x0.float().cpu().numpy(), y.double().cpu().numpy(),
                                 post_weight=w[1].double().cpu().numpy(), scale=0.5)
        got = x.double().cpu().numpy()
        assert (np.abs(got - xr) <= 2.0 ** -8 * np.abs(xr) + 1e-5).all()


@pytest.mark.gpu
@pytest.mark.parametrize("fmt", ["bf16", "fp8", "nvfp4"])
@pytest.mark.parametrize("T", [4, 5, 9, 16])
def test_both_ways_captured(fmt, T):
    """The two kernels and the two calls, whichever the batch takes: captured and
    replayed on new tokens with eager work between, the same bits as the eager
    call's, in a workspace full of NaN."""
    L = layer(FULL)
    bank = L.bank(fmt)
    x = synth.make_tokens(T, FULL).cuda()
    ws = moe.layer_few_workspace(L.ld, fmt, T)
    ws.fill_(255)
    y, ids, gates = [t.clone() for t in moe.layer_few(x, L.router, bank, L.ld, ws=ws)]
    i2, g2 = moe.route(x, L.router, L.ld)
    assert torch.equal(ids, i2)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        moe.layer_few(x, L.router, bank, L.ld, y=y, ids=ids, gates=gates, ws=ws)
    for k in range(3):
        x.copy_(torch.roll(synth.make_tokens(T + k, FULL)[:T], k + 1, 1))
        want = [t.clone() for t in moe.layer_few(x, L.router, bank, L.ld)]
        y.fill_(float("nan"))
        g.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip((y, ids, gates), want))


@pytest.mark.gpu
@pytest.mark.parametrize("T", [3, 16])
@pytest.mark.parametrize("fmt,e", [("fp8", -62), ("fp8", -67), ("nvfp4", -58), ("nvfp4", -59)])
def test_tiny_intermediate(fmt, e, T):
    """Tokens of about 2^e, so that the intermediate (about 2^2e; a block of it
    2^-16 of that) has a scale whose reciprocal is past the range of fp32: it
    counts as zero, in both ways alike, and y is finite."""
    L = layer(SMALL)
    up = L.up.clone()
    up[:, 16:32] *= 2.0 ** -8
    dev = moe.quantize_experts(up.cuda(), L.down_d, fmt, L.ld)
    x = (synth.make_tokens(T, SMALL).float() * 2.0 ** e).bfloat16()
    y, ids, gates = moe.layer_few(x.cuda(), L.router, dev, L.ld)
    i2, g2 = moe.route(x.cuda(), L.router, L.ld)
    assert torch.equal(ids, i2)
    y2 = moe.forward(x.cuda(), i2, g2, dev, L.ld)
    bank = om.ExpertBank(up, L.down, fmt).preload(np.unique(ids.cpu().numpy()), threads=8)
    ref, a = om.forward(x.float().numpy(), ids.cpu().numpy(), gates.double().cpu().numpy(), bank, return_a=True)
    rms = np.sqrt(np.mean(ref ** 2))
    print(f"{fmt} 2^{e} T={T}: amax of a {a.max():.2e} rms of y {rms:.2e} NaN {int(y.isnan().sum())}", flush=True)
    # the product of the intermediate's and the weights' scale is subnormal, with
    # 10 bits and more: inside TOL
    assert np.abs(y.double().cpu().numpy() - ref).max() <= TOL[fmt] * rms
    assert np.abs(y2.double().cpu().numpy() - ref).max() <= TOL[fmt] * rms


@pytest.mark.gpu
@pytest.mark.parametrize("fmt", ["bf16", "fp8", "nvfp4"])
@pytest.mark.parametrize("T", [1, 5, 12, 16])
def test_output_over_the_tokens(fmt, T):
    """y in place of x, and fp32 y whose first or last half is x: the bits of a
    call with buffers apart, every time."""
    L = layer(FULL)
    bank, n = L.bank(fmt), T * 2688
    x = synth.make_tokens(T, FULL).cuda()
    want = {t: moe.layer_few(x, L.router, bank, L.ld, y_dtype=t)[0] for t in (torch.bfloat16, torch.float32)}
    for _ in range(5):
        a = x.clone()
        y, ids, gates = moe.layer_few(a, L.router, bank, L.ld, y=a, y_dtype=torch.bfloat16)
        assert y is a and torch.equal(a, want[torch.bfloat16])
        for at in (0, n):
            store = torch.empty(n, device="cuda")
            a = store.view(torch.bfloat16)[at:at + n].view(T, 2688)
            a.copy_(x)
            moe.layer_few(a, L.router, bank, L.ld, y=store.view(T, 2688))
            assert torch.equal(store.view(T, 2688), want[torch.float32])


def _bank_of(fmt, dims, device="meta"):
    """A bank's tensors as quantize_experts lays them out, without data."""
    E, F, H = dims.n_experts, dims.ffn, dims.hidden
    e = lambda *shape, dtype=torch.uint8: torch.empty(shape, dtype=dtype, device=device)
    if fmt == "bf16":
        return moe.ExpertBank(fmt, e(E, F, H, dtype=torch.bfloat16), e(E, H, F, dtype=torch.bfloat16))
    s = lambda *shape: e(E, *shape, dtype=torch.float32)
    if fmt == "fp8":
        return moe.ExpertBank(fmt, e(E, F, H), e(E, H * F), None, None, s(), s())
    if fmt == "nvfp4":
        return moe.ExpertBank(fmt, e(E, F * H // 2), e(E, H * F // 2), e(E, F * H // 16), e(E, H * F // 16), s(), s())
    kh, kf = -(-H // 128), -(-F // 128)
    return moe.ExpertBank(fmt, e(E, moe.block_packed_size(F, H)), e(E, moe.block_packed_size(H, F)), None, None,
                          s(kf, kh), s(kh, kf))


@pytest.mark.parametrize("fmt", ["bf16", "fp8", "nvfp4", "fp8_block"])
def test_bank_of_other_dims_is_refused(fmt):
    """Every tensor of a bank is looked at: its size against the dims, its type where
    it is fixed, its device and layout.  (On the meta device: nothing is read.)"""
    dims, dev = moe.LayerDims(192, 320, 16, 2), torch.device("meta")
    good = _bank_of(fmt, dims)
    moe._check_bank(good, dims, dev)
    moe._check_bank(_bank_of(fmt, moe.LayerDims(192, 320, 32, 2)), dims, dev)  # its first experts
    names = [n for n in ("up", "down", "up_bs", "down_bs", "up_s", "down_s") if getattr(good, n) is not None]
    assert len(names) == {"bf16": 2, "fp8": 4, "nvfp4": 6, "fp8_block": 4}[fmt]
    for n in names:
        t = getattr(good, n)
        bad = [t[:15], None, torch.empty_like(t, device="cpu"), torch.empty((2,) + t.shape, dtype=t.dtype, device=dev)[:, :8]]
        if t.dtype != torch.uint8:
            bad += [t.to(torch.float64)]
        for b in bad:
            bank = _bank_of(fmt, dims)
            setattr(bank, n, b)
            with pytest.raises(ValueError, match=n):
                moe._check_bank(bank, dims, dev)
    for other in (moe.LayerDims(256, 320, 16, 2), moe.LayerDims(192, 384, 16, 2), moe.LayerDims(192, 320, 32, 2)):
        with pytest.raises(ValueError):
            moe._check_bank(good, other, dev)


@pytest.mark.gpu
@pytest.mark.parametrize("fmt", ["bf16", "fp8", "nvfp4", "fp8_block"])
def test_wrong_banks_and_biases_are_refused(fmt):
    """The call itself: refused on the host, nothing is launched."""
    L = layer(SMALL)
    x = synth.make_tokens(3, SMALL).cuda()
    small = _bank_of(fmt, moe.LayerDims(256, 192, 16, 4), "cuda")
    with pytest.raises(ValueError, match="up"):
        moe.layer_few(x, L.router, small, L.ld)
    for bias in (L.router.bias[:16], L.router.bias.double(), L.router.bias.cpu()):
        with pytest.raises(ValueError, match="bias"):
            moe.layer_few(x, moe.PackedRouter(L.router.w_packed, bias), L.bank(fmt), L.ld)


@pytest.mark.gpu
@pytest.mark.parametrize("fmt", ["bf16", "fp8", "nvfp4"])
@pytest.mark.parametrize("T", [1, 6])
def test_more_column_tiles_than_workgroups(fmt, T):
    """H = 8192: 512 tiles of the down projection for 256 workgroups, two each."""
    d = synth.Dims(hidden=8192, ffn=192, n_experts=16, top_k=3)
    check(layer(d), fmt, synth.make_tokens(T, d))
