"""The 8-bit state cache (gma_state_store, gma_state_load): codes, scales and values are those of the format, bit by bit."""
import ctypes

import numpy as np
import pytest

from oracle import delta as ref

torch = pytest.importorskip("torch")
gpu = pytest.mark.gpu


@pytest.fixture(scope="module")
def gma():
    import __graft_entry__
    __graft_entry__.build()
    import gaussian_mixture_latent_gb300 as m
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    return m


def test_format_error_is_at_most_half_a_step():
    x = (np.random.RandomState(0).randn(50, 65) * np.exp(np.random.RandomState(1).randn(50, 1))).astype(np.float32)
    codes, scales = ref.quantise(x)
    y = ref.dequantise(codes, scales)
    step = np.repeat(scales, 32, axis=-1)[:, :65]
    # half a step, and the roundings of the quotient and the product (2^-24 of up to 127 steps each)
    assert (np.abs(x - y) <= step * (0.5 + 2 * 127 * 2.0 ** -24)).all()
    # a group of one value: code 127, so 127 scale with scale = x (1 / 127): the constant, its product with x and the
    # product with 127 round once each
    assert np.abs(x[:, 64] - y[:, 64]).max() <= 3 * 2.0 ** -24 * np.abs(x[:, 64]).max()


def test_refusals_through_the_c_interface():
    import __graft_entry__
    __graft_entry__.build()
    import gaussian_mixture_latent_gb300 as m
    from gaussian_mixture_latent_gb300 import delta
    lib = delta._lib()
    p, odd = ctypes.c_void_p(4096), ctypes.c_void_p(4100)

    def call(f, ws=p, wsb=256, at=None, val=None, **kw):
        d = m.gma_state_desc(**dict(dict(n=2, n_states=3, n_cache=4, rows=8, cols=16), **kw))
        args = [p] * 5
        if at is not None:
            args[at] = val
        return f(ctypes.byref(d), *args, ws, wsb, None)

    for f, index in ((lib.gma_state_store, (1, 2)), (lib.gma_state_load, (2, 3))):
        for bad in (dict(n=-1), dict(n_states=0), dict(n_cache=-2), dict(rows=0), dict(cols=0)):
            assert call(f, **bad) == 1, bad
        for i in range(5):
            assert call(f, at=i, val=odd) == 1
            if i not in index:
                assert call(f, at=i, val=None) == 1
        for i in index:
            assert call(f, at=i, val=None, n=4) == 1       # entry i at i: not within three states
        assert call(f, rows=1 << 20, cols=1 << 20) == 2 and call(f, n=70000) == 2
        assert call(f, ws=None) == 3 and call(f, wsb=8) == 3 and call(f, n=0) == 0
        assert f(None, p, p, p, p, p, p, 256, None) == 1


def pools(S, P, H, R, C, seed=0):
    gen = torch.Generator().manual_seed(seed)
    state = torch.randn((S, H, R, C), generator=gen) * torch.exp(2 * torch.randn((S, H, R, 1), generator=gen))
    codes = torch.randint(-127, 128, (P, H, R, C), generator=gen, dtype=torch.int8)
    scales = torch.rand((P, H, R, -(-C // 32)), generator=gen)
    return state, codes, scales


@gpu
@pytest.mark.parametrize("H,R,C", [(1, 1, 1), (2, 3, 5), (3, 7, 31), (2, 5, 32), (2, 4, 33), (12, 64, 65), (4, 128, 128),
                                   (2, 9, 80), (2, 16, 129), (1, 64, 64), (3, 200, 256)])
def test_store_and_load(gma, H, R, C):
    state, codes, scales = pools(6, 5, H, R, C)
    src, dst = torch.tensor([5, -1, 0, 3], dtype=torch.int32), torch.tensor([1, 2, 4, -1], dtype=torch.int32)
    st, co, sc = state.cuda(), codes.cuda(), scales.cuda()
    got = gma.gma_state_store(st, co, sc, src=src.cuda(), dst=dst.cuda(), check_status=True)
    assert got[0] is co and got[1] is sc
    for i, j in ((5, 1), (0, 4)):
        q, s = ref.quantise(state[i].numpy())
        assert np.array_equal(co[j].cpu().numpy(), q) and np.array_equal(sc[j].cpu().numpy(), s)
    for j in (0, 2, 3):
        assert torch.equal(co[j].cpu(), codes[j]) and torch.equal(sc[j].cpu(), scales[j])
    assert torch.equal(st.cpu(), state)
    back = gma.gma_state_load(co, sc, st, src=torch.tensor([4, 0, -3, 4], dtype=torch.int32).cuda(),
                              dst=torch.tensor([2, 0, 1, 5], dtype=torch.int32).cuda(), check_status=True)
    assert back is st
    for i, j in ((4, 2), (0, 0), (4, 5)):
        want = ref.dequantise(co[i].cpu().numpy(), sc[i].cpu().numpy())
        assert np.array_equal(st[j].cpu().numpy(), want)
    for j in (1, 3, 4):
        assert torch.equal(st[j].cpu(), state[j])


@gpu
def test_values_out_of_the_ordinary(gma):
    x = torch.randn(1, 1, 8, 96)
    x[0, 0, 0, 3] = float("nan")
    x[0, 0, 1, 40] = float("inf")
    x[0, 0, 2, 95] = -float("inf")
    x[0, 0, 3] = 0.0
    x[0, 0, 4] *= 1e-43                                   # subnormal: the scale is one too, or zero
    x[0, 0, 5] = 1e-45
    x[0, 0, 6] *= 1e38
    x[0, 0, 7, ::2] = 0.5
    codes, scales = torch.zeros(1, 1, 8, 96, dtype=torch.int8).cuda(), torch.zeros(1, 1, 8, 3).cuda()
    back = torch.zeros_like(x).cuda()
    gma.gma_state_store(x.cuda(), codes, scales)
    gma.gma_state_load(codes, scales, back)
    q, s = ref.quantise(x.numpy())
    assert np.array_equal(codes.cpu().numpy(), q) and np.array_equal(scales.cpu().numpy(), s, equal_nan=True)
    assert np.array_equal(back.cpu().numpy(), ref.dequantise(q, s), equal_nan=True)
    bad = torch.isnan(back.cpu()).reshape(8, 3, 32).all(-1)
    assert bad.sum() == 3 and bad[0, 0] and bad[1, 1] and bad[2, 2]
    assert torch.isnan(back).sum() == 96


@gpu
def test_the_same_destination_twice_and_bad_indices(gma):
    state, codes, scales = pools(6, 5, 2, 16, 64, seed=3)
    st, co, sc = state.cuda(), codes.cuda(), scales.cuda()
    t = lambda *v: torch.tensor(v, dtype=torch.int32).cuda()
    gma.gma_state_store(st, co, sc, src=t(0, 1, 2, 3), dst=t(3, 1, 3, 1), check_status=True)
    for i, j in ((2, 3), (3, 1)):                         # the last entry counts
        q, s = ref.quantise(state[i].numpy())
        assert np.array_equal(co[j].cpu().numpy(), q) and np.array_equal(sc[j].cpu().numpy(), s)
    before = co.clone(), sc.clone(), st.clone()
    for a, b in ((t(6, 0), t(0, 5)), (t(2 ** 31 - 1, -2 ** 31), t(0, 0))):
        with pytest.raises(gma.GmaError) as e:
            gma.gma_state_store(st, co, sc, src=a, dst=b, check_status=True)
        assert e.value.code == 6
    with pytest.raises(gma.GmaError):
        gma.gma_state_load(co, sc, st, src=t(5, 0), dst=t(0, 6), check_status=True)
    assert torch.equal(co, before[0]) and torch.equal(sc, before[1]) and torch.equal(st, before[2])
    # an entry that copies nothing does not hide an earlier one with its destination
    gma.gma_state_store(st, co, sc, src=t(4, -1), dst=t(0, 0), check_status=True)
    q, s = ref.quantise(state[4].numpy())
    assert np.array_equal(co[0].cpu().numpy(), q)


@gpu
def test_defaults_refusals_and_graph(gma):
    state, codes, scales = (x.cuda() for x in pools(3, 4, 2, 32, 65, seed=5))
    want = ref.quantise(state.cpu().numpy())
    g = torch.cuda.CUDAGraph()
    gma.gma_state_store(state, codes, scales)
    torch.cuda.synchronize()
    assert np.array_equal(codes[:3].cpu().numpy(), want[0])
    codes.zero_()
    with torch.cuda.graph(g):
        gma.gma_state_store(state, codes, scales)
    state.mul_(3.0)
    g.replay()
    torch.cuda.synchronize()
    assert np.array_equal(codes[:3].cpu().numpy(), ref.quantise(state.cpu().numpy())[0])
    with pytest.raises(ValueError):
        gma.gma_state_store(state, codes.int(), scales)
    with pytest.raises(ValueError):
        gma.gma_state_store(state, codes, scales[..., :2].contiguous())
    with pytest.raises(ValueError):
        gma.gma_state_load(codes, scales, state.transpose(2, 3))
    with pytest.raises(ValueError):
        gma.gma_state_load(codes, scales, state, src=torch.zeros(2, dtype=torch.int32, device="cuda"),
                           dst=torch.zeros(3, dtype=torch.int32, device="cuda"))


@gpu
def test_mixture_memories_of_gma_decode(gma):
    """The causal mixture's [K, dv + 1] memories parked and resumed: the decode that follows sees them within the
    format's error."""
    from gaussian_mixture_latent_gb300 import inputs
    from tests._util import to_device
    w = inputs.Workload("park", B=2, H=2, N=60, d=64, K=64, dv=64, dtype="bf16", causal=True, seed=3)
    x = inputs.gen_all(w)
    y = {n: to_device(x[n]) for n in ("Qx", "Kx", "V", "mu", "rho", "alpha")}
    par = (y["mu"], y["rho"], y["alpha"])
    cut = lambda a, b: [y[n][:, :, a:b].contiguous() for n in ("Qx", "Kx", "V")]
    state = torch.zeros((2, 2, 64, 65), device="cuda")
    gma.gma_decode(*cut(0, 50), *par, state)
    codes = torch.zeros(state.shape, dtype=torch.int8, device="cuda")
    scales = torch.zeros((2, 2, 64, 3), device="cuda")
    gma.gma_state_store(state, codes, scales)
    back = gma.gma_state_load(codes, scales, torch.empty_like(state))
    # the normaliser column is a group of its own: the constant, the scale and the product round once each
    assert (back[..., 64] - state[..., 64]).abs().max() <= 3 * 2.0 ** -24 * state[..., 64].abs().max()
    step = scales[..., :2].repeat_interleave(32, -1)
    assert ((back[..., :64] - state[..., :64]).abs() <= step * (0.5 + 2 * 127 * 2.0 ** -24)).all()
    # a read is sum gamma V / sum gamma Z: no memory row adds more than (its error) / (its Z), and new rows only
    # add to Z; the two bf16 outputs round once each
    worst = (0.5 * scales[..., :2].amax(-1) / state[..., 64]).max().item()
    a, b = gma.gma_decode(*cut(50, 60), *par, state), gma.gma_decode(*cut(50, 60), *par, back)
    assert (a.float() - b.float()).abs().max().item() <= worst + 2 * 2.0 ** -8 * a.float().abs().max().item()
