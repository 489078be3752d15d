"""The gated delta rule (gma_delta_forward, _backward, _decode) against its float64 recurrence.

Tolerances are of the largest error of a tensor over its largest value.
float32: a row's sums have d + 4 roundings of 2^-24 and the recurrence does not amplify them (|I - beta k k^T| <= 1,
decay <= 1), so N rows leave about sqrt(N (d + 4)) 2^-24; eight times that for the maximum over all elements.  The
gradients' running sums over a chunk add as many terms again: twice that.
bfloat16: half a step (2^-8) for the rounding of the result, and as much for each of the two intermediates that a
bf16 path may hold in one bf16 term (the state and u of the output's products); gradients have one more (dO's or x's
products with the states).  States in float32 come from three-term products: the float32 bound with the terms of a
64-row chunk's inverse counted again (a factor of 4).
"""
import numpy as np
import pytest

from oracle import delta as ref

torch = pytest.importorskip("torch")
gpu = pytest.mark.gpu
DT = {"f32": torch.float32, "bf16": torch.bfloat16}


@pytest.fixture(scope="module")
def gma():
    import __graft_entry__
    __graft_entry__.build()
    import gaussian_mixture_latent_gb300 as m
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    return m


def tol32(N, d):
    return 8 * (max(N, 1) * (d + 4)) ** 0.5 * 2.0 ** -24


def make(B, H, N, d, dv, dtype="f32", gates="f32", Hk=None, seed=0, state=False, lengths=None, rate=0.3):
    """Inputs on the CPU, as tensors of their types."""
    gen = torch.Generator().manual_seed(seed)
    n = lambda *s: torch.randn(s, generator=gen)
    unit = lambda x: x / x.norm(dim=-1, keepdim=True)
    Hk = Hk or H
    x = dict(Qx=unit(n(B, Hk, N, d)).to(DT[dtype]), Kx=unit(n(B, Hk, N, d) + 0.5 * n(B, Hk, 1, d)).to(DT[dtype]),
             V=n(B, H, N, dv).to(DT[dtype]), g=(-rate * torch.rand((B, H, N), generator=gen)).to(DT[gates]),
             beta=torch.sigmoid(n(B, H, N)).to(DT[gates]))
    x["state"] = n(B, H, d, dv) if state else None
    x["dstate"] = n(B, H, d, dv) if state else None
    x["dO"] = n(B, H, N, dv).to(DT[dtype])
    x["lengths"] = None if lengths is None else torch.tensor(lengths, dtype=torch.int32)
    return x


def f64(t):
    return None if t is None else t.detach().to(torch.float64).cpu().numpy()


def cuda(x):
    return {k: v.cuda() if isinstance(v, torch.Tensor) else v for k, v in x.items()}


ARGS = ("Qx", "Kx", "V", "g", "beta")


def reference(x, scale=None):
    scale = x["Qx"].shape[-1] ** -0.5 if scale is None else scale
    with np.errstate(invalid="ignore"):
        return ref.forward(*(f64(x[n]) for n in ARGS), scale, f64(x["state"]),
                           None if x["lengths"] is None else x["lengths"].numpy())


def reference_grads(x, scale=None):
    scale = x["Qx"].shape[-1] ** -0.5 if scale is None else scale
    with np.errstate(invalid="ignore"):
        return ref.backward(*(f64(x[n]) for n in ARGS), scale, f64(x["dO"]), f64(x["state"]), f64(x["dstate"]),
                            None if x["lengths"] is None else x["lengths"].numpy())


def off(got, want):
    got = f64(got)
    assert got.shape == want.shape
    assert np.isfinite(got).all()
    if got.size == 0:
        return 0.0
    big = np.abs(want).max()
    return np.abs(got - want).max() / big if big else np.abs(got).max()


# ------------------------------------------------------------------------------------------ CPU: the reference itself

def test_reference_gradient_against_differences():
    x = make(1, 2, 7, 3, 2, Hk=1, seed=3, state=True, lengths=[6])
    a = {n: f64(x[n]) for n in ARGS + ("state",)}
    dO, dS, ln = f64(x["dO"]), f64(x["dstate"]), np.array([6])

    def loss(**kw):
        y = dict(a, **kw)
        o, S = ref.forward(*(y[n] for n in ARGS), 0.7, y["state"], ln)
        return (o * dO).sum() + (S * dS).sum()

    grads = dict(zip(ARGS + ("state",), ref.backward(*(a[n] for n in ARGS), 0.7, dO, a["state"], dS, ln)))
    for name, gr in grads.items():
        flat = np.zeros(a[name].size)
        for i in range(flat.size):
            hi, lo = a[name].copy(), a[name].copy()
            hi.flat[i] += 1e-5
            lo.flat[i] -= 1e-5
            flat[i] = (loss(**{name: hi}) - loss(**{name: lo})) / 2e-5
        # central differences: h^2 times the third derivative, and 2^-53 / h
        assert np.abs(flat - gr.ravel()).max() <= 1e-8 * max(1.0, np.abs(gr).max()), name


def test_reference_of_identical_keys_keeps_the_last_value():
    # beta = 1, no decay, one unit key: the state holds exactly the last value under that key
    x = make(1, 1, 5, 4, 3)
    x["Kx"][:] = torch.tensor([1.0, 0, 0, 0])
    x["Qx"][:] = torch.tensor([1.0, 0, 0, 0])
    x["g"][:], x["beta"][:] = 0.0, 1.0
    out, S = reference(x, 1.0)
    assert np.allclose(out, f64(x["V"]), atol=1e-15) and np.allclose(S[0, 0, 0], f64(x["V"])[0, 0, -1], atol=1e-15)


# ------------------------------------------------------------------------------------------ CPU: refusals

def test_refusals_through_the_c_interface():
    import ctypes

    import __graft_entry__
    __graft_entry__.build()
    import gaussian_mixture_latent_gb300 as m
    from gaussian_mixture_latent_gb300 import delta
    lib = delta._lib()
    p, odd, n = ctypes.c_void_p(4096), ctypes.c_void_p(4100), ctypes.c_size_t(0)

    def desc(**kw):
        base = dict(B=2, H=4, Hk=2, N=100, d=64, dv=64, in_dtype=1, gate_dtype=0, scale=0.125)
        return m.gma_delta_desc(**dict(base, **kw))

    sizes = (lib.gma_delta_workspace_size, lib.gma_delta_backward_workspace_size, lib.gma_delta_decode_workspace_size)
    for f in sizes:
        assert f(ctypes.byref(desc()), ctypes.byref(n)) == 0 and n.value >= 256
        assert f(None, ctypes.byref(n)) == 1 and f(ctypes.byref(desc()), None) == 1
        for bad in (dict(B=0), dict(H=0), dict(Hk=0), dict(Hk=3), dict(N=-1), dict(d=0), dict(dv=-4), dict(in_dtype=2),
                    dict(gate_dtype=9), dict(scale=float("nan")), dict(scale=float("inf"))):
            assert f(ctypes.byref(desc(**bad)), ctypes.byref(n)) == 1, bad
        for far in (dict(d=257), dict(dv=300), dict(B=65536, H=2, Hk=2), dict(N=2 ** 31 - 1)):
            assert f(ctypes.byref(desc(**far)), ctypes.byref(n)) == 2, far

    def call(f, count, need, d=None, tail=None, **at):
        args = [p] * count
        for i, v in at.items():
            args[int(i[1:])] = v
        return f(ctypes.byref(d or desc()), *args, *(tail or (p, need, None)))

    big = 1 << 40
    for i in (0, 1, 2, 3, 4, 7):                          # Qx, Kx, V, g, beta, out
        assert call(lib.gma_delta_forward, 9, big, **{f"a{i}": None}) == 1
    for i in range(9):
        assert call(lib.gma_delta_forward, 9, big, **{f"a{i}": odd}) == 1
    assert call(lib.gma_delta_forward, 9, 0, tail=(None, big, None)) == 3
    assert call(lib.gma_delta_forward, 9, 16) == 3
    assert call(lib.gma_delta_forward, 9, big, d=desc(N=0), a8=None) == 0
    for i in (0, 1, 2, 3, 4, 7, 9, 10, 11, 12, 13):
        assert call(lib.gma_delta_backward, 15, big, **{f"a{i}": None}) == 1
    for i in range(15):
        assert call(lib.gma_delta_backward, 15, big, **{f"a{i}": odd}) == 1
    assert call(lib.gma_delta_backward, 15, 256) == 3
    assert call(lib.gma_delta_backward, 15, big, d=desc(N=0), a14=None) == 0

    def dec(d=None, n_states=8, slots=p, ws=p, wsb=256, **at):
        args = [p] * 5
        for i, v in at.items():
            args[int(i[1:])] = v
        return lib.gma_delta_decode(ctypes.byref(d or desc()), *args, None, slots, n_states, at.get("state", p) if
                                    "state" in at else p, p, ws, wsb, None)

    assert dec(n_states=0) == 1 and dec(n_states=1, slots=None) == 1 and dec(a0=None) == 1 and dec(slots=odd) == 1
    assert dec(ws=None) == 3 and dec(wsb=255) == 3 and dec(d=desc(N=0)) == 0 and dec(d=desc(d=300)) == 2


def test_sizes_beyond_the_c_interface_are_refused():
    from gaussian_mixture_latent_gb300 import GmaError, delta
    delta._sizes("x", 1, 2 ** 31 - 1)
    with pytest.raises(GmaError) as e:
        delta._sizes("x", 1, 2 ** 32 + 8)
    assert e.value.code == 2


@pytest.mark.parametrize("what", ["forward", "backward", "decode"])
def test_python_refusals_on_cpu_tensors(what):
    import gaussian_mixture_latent_gb300 as m
    x = make(1, 2, 4, 8, 8)
    args = [x[n] for n in ARGS]
    with pytest.raises(ValueError):
        if what == "forward":
            m.gma_delta_forward(*args)
        elif what == "backward":
            m.gma_delta_backward(*args, x["dO"])
        else:
            m.gma_delta_decode(*args, torch.zeros(1, 2, 8, 8))


# ------------------------------------------------------------------------------------------ GPU: forward

SHAPES = [
    # B, H, Hk, N, d, dv
    (1, 1, 1, 1, 1, 1), (2, 3, 3, 2, 5, 7), (1, 2, 1, 9, 16, 33), (2, 4, 2, 31, 64, 64), (1, 2, 2, 32, 64, 128),
    (2, 2, 1, 33, 128, 64), (1, 4, 4, 63, 128, 128), (3, 2, 2, 64, 64, 64), (1, 4, 1, 65, 96, 80), (1, 2, 2, 127, 100, 36),
    (2, 2, 2, 130, 128, 128), (1, 1, 1, 150, 256, 256), (1, 3, 3, 301, 64, 64), (1, 2, 2, 257, 32, 48), (1, 1, 1, 200, 8, 136),
    (2, 2, 1, 190, 200, 64), (1, 2, 2, 191, 128, 200),
]


def run_forward(m, x, **kw):
    y = cuda(x)
    r = m.gma_delta_forward(*(y[n] for n in ARGS), state=y["state"], lengths=y["lengths"], return_state=True,
                            check_status=True, **kw)
    plain = m.gma_delta_forward(*(y[n] for n in ARGS), state=y["state"], lengths=y["lengths"], check_status=True, **kw)
    return r[0], r[1], plain


def check_forward(m, x, dtype, **kw):
    B, Hk, N, d = x["Qx"].shape
    want, S = reference(x, **kw)
    out, state, plain = run_forward(m, x, **kw)
    t = tol32(N, d)
    tout = t if dtype == "f32" else 3 * 2.0 ** -8
    assert off(out, want) <= tout and off(plain, want) <= tout
    assert off(state, S) <= (t if dtype == "f32" else 4 * t)


@gpu
@pytest.mark.parametrize("dtype,gates", [("f32", "f32"), ("bf16", "f32"), ("bf16", "bf16"), ("f32", "bf16")])
@pytest.mark.parametrize("shape", SHAPES, ids=str)
def test_forward(gma, shape, dtype, gates):
    B, H, Hk, N, d, dv = shape
    x = make(B, H, N, d, dv, dtype, gates, Hk=Hk, seed=N + d, state=(N % 2 == 1))
    check_forward(gma, x, dtype)


# heads and dv from one CTA to 16 columns to one to 64, at both widths: the same rule as a few heads, and for the backward
MANY = [(2, 20, 10, 150, 64, 64), (3, 30, 30, 130, 64, 128), (5, 8, 4, 140, 128, 128), (3, 10, 10, 200, 128, 128),
        (1, 90, 90, 100, 128, 64), (2, 25, 25, 129, 96, 72), (3, 25, 25, 70, 48, 200)]


@gpu
@pytest.mark.parametrize("gates", ["f32", "bf16"])
@pytest.mark.parametrize("shape", MANY, ids=str)
def test_many_heads(gma, shape, gates):
    B, H, Hk, N, d, dv = shape
    lengths = [N, N - 37, 0, 64, 1][:B]
    check_forward(gma, make(B, H, N, d, dv, "bf16", gates, Hk=Hk, seed=N, state=True, lengths=lengths), "bf16")
    check_backward(gma, make(B, H, N, d, dv, "bf16", gates, Hk=Hk, seed=N, state=True, lengths=lengths), "bf16", gates)
    check_backward(gma, make(B, H, N, d, dv, "bf16", gates, Hk=Hk, seed=N + 1), "bf16", gates)


@gpu
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("d,dv", [(64, 64), (128, 128), (24, 20)])
def test_forward_of_a_padded_batch(gma, d, dv, dtype):
    lengths = [0, 1, 63, 64, 65, 150, 151, -4, 400]
    N = 151
    x = make(len(lengths), 2, N, d, dv, dtype, lengths=lengths, seed=5, state=True)
    dead = torch.arange(N)[None] >= torch.tensor(lengths)[:, None]
    for n in ARGS:                                        # what padding holds is not used
        t = x[n]
        t[(dead[:, None] if t.dim() == 3 else dead[:, None, :, None]).expand(t.shape)] = float("nan")
    x["V"][3, 0, 149, 0] = float("inf")
    check_forward(gma, x, dtype)
    out, state, _ = run_forward(gma, x)
    for b in (0, 7):                                      # nothing there: zeros out, the state as it was
        assert not out[b].any() and torch.equal(state[b].cpu(), x["state"][b])


@gpu
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("low", [float("-inf"), -1e4, torch.finfo(torch.float32).min])
@pytest.mark.parametrize("d,dv", [(64, 64), (128, 64), (17, 6)])
def test_forward_resets(gma, d, dv, low, dtype):
    # a decay of zero forgets the state: the rows after it do not see the rows before, in or out of a chunk
    x = make(1, 2, 200, d, dv, dtype, seed=9, state=True)
    for t in (0, 5, 6, 63, 64, 130, 199):
        x["g"][:, 0, t] = low
    check_forward(gma, x, dtype)


@gpu
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_forward_special_gates(gma, dtype):
    # beta = 0 everywhere in one head (the state only fades), beta = 1 with identical keys in the other
    x = make(1, 2, 140, 64, 64, dtype, seed=4, state=True)
    x["beta"][:, 0], x["beta"][:, 1] = 0.0, 1.0
    x["Kx"][:, 1] = 0.0
    x["Kx"][:, 1, :, 3] = 1.0
    x["g"][:, 1] = 0.0
    check_forward(gma, x, dtype)
    check_forward(gma, x, dtype, scale=1.75)


@gpu
def test_forward_of_strong_and_weak_decay(gma):
    for rate in (0.0, 1e-4, 3.0, 40.0):
        check_forward(gma, make(1, 3, 300, 64, 64, "bf16", seed=11, state=True, rate=rate), "bf16")


@gpu
@pytest.mark.parametrize("size", [1e-6, 1e5, 1e30])
def test_forward_of_small_and_large_values(gma, size):
    x = make(1, 2, 100, 64, 64, "bf16", seed=12)
    x["V"] = (x["V"].float() * size).to(torch.bfloat16)
    check_forward(gma, x, "bf16")


@gpu
def test_forward_in_pieces_is_the_forward_of_the_whole(gma):
    x = cuda(make(2, 4, 333, 128, 128, "bf16", Hk=2, seed=13, state=True))
    whole, S = gma.gma_delta_forward(*(x[n] for n in ARGS), state=x["state"], return_state=True)
    state, outs = x["state"].clone(), []
    for a, b in ((0, 1), (1, 100), (100, 228), (228, 333)):
        part = [x[n][:, :, a:b].contiguous() for n in ARGS]
        o, same = gma.gma_delta_forward(*part, state=state, state_out=state)
        assert same is state
        outs.append(o)
    assert off(torch.cat(outs, 2), f64(whole)) <= 6 * 2.0 ** -8 and off(state, f64(S)) <= 8 * tol32(333, 128)


@gpu
def test_forward_empty(gma):
    x = cuda(make(2, 2, 0, 64, 64, "bf16", state=True))
    out, S = gma.gma_delta_forward(*(x[n] for n in ARGS), state=x["state"], return_state=True)
    assert out.shape == (2, 2, 0, 64) and torch.equal(S, x["state"])
    out, S = gma.gma_delta_forward(*(x[n] for n in ARGS), return_state=True)
    assert not S.any()


# ------------------------------------------------------------------------------------------ GPU: backward

NAMES = ("dQx", "dKx", "dV", "dg", "dbeta", "dstate")


def check_backward(m, x, dtype, gates, **kw):
    B, Hk, N, d = x["Qx"].shape
    want = reference_grads(x, **kw)
    y = cuda(x)
    got = m.gma_delta_backward(*(y[n] for n in ARGS), y["dO"], state=y["state"], dstate=y["dstate"],
                               lengths=y["lengths"], check_status=True, **kw)
    t = 2 * tol32(N, d)
    for name, a, b in zip(NAMES, got, want):
        if name == "dstate":
            if y["state"] is not None:
                assert off(a, b) <= (t if dtype == "f32" else 4 * t), name
            continue
        assert a.dtype == y[dict(dQx="Qx", dKx="Kx", dV="V", dg="g", dbeta="beta")[name]].dtype
        if dtype == "f32":
            # dg and dbeta in bf16 are rounded once
            lim = t + (2.0 ** -8 if gates == "bf16" and name in ("dg", "dbeta") else 0)
        else:
            lim = 4 * 2.0 ** -8
        assert off(a, b) <= lim, (name, off(a, b), lim)
    return got


@gpu
@pytest.mark.parametrize("dtype,gates", [("f32", "f32"), ("bf16", "f32"), ("bf16", "bf16"), ("f32", "bf16")])
@pytest.mark.parametrize("shape", SHAPES, ids=str)
def test_backward(gma, shape, dtype, gates):
    B, H, Hk, N, d, dv = shape
    check_backward(gma, make(B, H, N, d, dv, dtype, gates, Hk=Hk, seed=N + d, state=(N % 2 == 1)), dtype, gates)


@gpu
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("d,dv", [(64, 64), (128, 128), (24, 20)])
def test_backward_of_a_padded_batch(gma, d, dv, dtype):
    lengths = [0, 1, 32, 64, 65, 150, 151, -4]
    N = 151
    x = make(len(lengths), 2, N, d, dv, dtype, Hk=1, lengths=lengths, seed=6, state=True)
    dead = torch.arange(N)[None] >= torch.tensor(lengths)[:, None]
    for n in ARGS + ("dO",):
        t = x[n]
        t[(dead[:, None] if t.dim() == 3 else dead[:, None, :, None]).expand(t.shape)] = float("nan")
    got = check_backward(gma, x, dtype, "f32")
    for t in got[:5]:                                     # exact zeros where there is no row
        hidden = t[(dead.cuda()[:, None] if t.dim() == 3 else dead.cuda()[:, None, :, None]).expand(t.shape)]
        assert not hidden.any()
    assert torch.equal(got[5][0].cpu(), x["dstate"][0])


@gpu
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("low", [float("-inf"), -1e4, torch.finfo(torch.float32).min])
def test_backward_resets(gma, low, dtype):
    x = make(1, 2, 150, 64, 64, dtype, seed=9, state=True)
    for t in (5, 6, 63, 64, 130, 149):
        x["g"][:, 0, t] = low
    got = check_backward(gma, x, dtype, "f32")
    for t in (5, 6, 63, 64, 130, 149):                    # nothing comes through a decay of zero
        assert not got[3][0, 0, t].any()


@gpu
def test_backward_special_gates(gma):
    for dtype in ("f32", "bf16"):
        x = make(1, 2, 100, 64, 64, dtype, seed=4, state=True)
        x["beta"][:, 0], x["beta"][:, 1] = 0.0, 1.0
        x["Kx"][:, 1] = 0.0
        x["Kx"][:, 1, :, 3] = 1.0
        x["g"][:, 1] = 0.0
        check_backward(gma, x, dtype, "f32", scale=0.6)


@gpu
def test_backward_against_differences_of_the_forward(gma):
    # directional central differences of the float32 forward: h = 2^-7 against sums of 2^-24 relative error
    x = make(1, 2, 70, 32, 16, seed=21, state=True)
    y = cuda(x)
    got = gma.gma_delta_backward(*(y[n] for n in ARGS), y["dO"], state=y["state"], dstate=y["dstate"])
    gen = torch.Generator().manual_seed(5)
    for name, gr in zip(ARGS + ("state",), got):
        way = torch.randn(y[name].shape, generator=gen).cuda()
        way = way / way.norm()

        def loss(h):
            z = dict(y, **{name: y[name] + h * way})
            o, S = gma.gma_delta_forward(*(z[n] for n in ARGS), state=z["state"], return_state=True)
            return ((o.double() * y["dO"].double()).sum() + (S.double() * y["dstate"].double()).sum()).item()

        h = 2.0 ** -7
        diff, dot = (loss(h) - loss(-h)) / (2 * h), (gr.double() * way.double()).sum().item()
        # rounding: |loss terms| (about sqrt(sum o^2 dO^2) ~ 50) * 2^-24 * 8 / h; curvature: h^2 |third derivative|
        assert abs(diff - dot) <= 50 * 2.0 ** -24 * 8 / h + 4 * h * h * max(1.0, abs(dot)) , name


@gpu
def test_backward_without_state_and_empty(gma):
    x = cuda(make(1, 2, 40, 64, 64, seed=2))
    got = gma.gma_delta_backward(*(x[n] for n in ARGS), x["dO"])
    assert got[5] is None
    y = cuda(make(1, 2, 0, 64, 64, state=True))
    got = gma.gma_delta_backward(*(y[n] for n in ARGS), y["dO"], state=y["state"], dstate=y["dstate"])
    assert torch.equal(got[5], y["dstate"]) and got[0].numel() == 0
    again = gma.gma_delta_backward(*(x[n] for n in ARGS), x["dO"])
    first = gma.gma_delta_backward(*(x[n] for n in ARGS), x["dO"])
    assert all(torch.equal(a, b) for a, b in zip(again[:5], first[:5]))


# ------------------------------------------------------------------------------------------ GPU: decode

@gpu
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("N", [1, 2, 5, 20])
@pytest.mark.parametrize("H,Hk,d,dv", [(12, 12, 64, 64), (4, 2, 128, 128), (2, 1, 40, 72), (2, 2, 256, 130), (1, 1, 3, 5),
                                       (2, 2, 96, 64)])
def test_decode(gma, H, Hk, d, dv, N, dtype):
    B, pool = 5, 9
    x = make(B, H, N, d, dv, dtype, Hk=Hk, seed=N + d)
    gen = torch.Generator().manual_seed(8)
    states = torch.randn((pool, H, d, dv), generator=gen)
    slots = torch.tensor([7, -1, 0, 3, 8], dtype=torch.int32)
    live = [0, 2, 3, 4]
    y = {n: (x[n][live] if isinstance(x[n], torch.Tensor) else None) for n in x}
    y["state"] = states[slots[live].long()]
    want, S = reference(y)
    z, st = cuda(x), states.cuda()
    out = gma.gma_delta_decode(*(z[n] for n in ARGS), st, slots=slots.cuda(), check_status=True)
    assert off(out[live], want) <= (tol32(N, d) if dtype == "f32" else 2.0 ** -8 + tol32(N, d))
    assert not out[1].any()
    assert off(st[slots[live].long().cuda()], S) <= tol32(N, d)
    for i in (1, 2, 4, 5, 6):                             # states that no entry names stay as they were
        assert torch.equal(st[i].cpu(), states[i])


@gpu
def test_decode_bad_slots(gma):
    x = cuda(make(4, 2, 1, 64, 64, seed=1))
    states = torch.randn((6, 2, 64, 64), device="cuda")
    st = states.clone()
    good = gma.gma_delta_decode(*(x[n] for n in ARGS), st, slots=torch.tensor([5, 1, 2, 3], dtype=torch.int32).cuda())
    for bad in ([5, 6, 2, 3], [5, 2 ** 31 - 1, 2, 3], [5, 5, 2, 3]):
        st2 = states.clone()
        with pytest.raises(gma.GmaError) as e:
            gma.gma_delta_decode(*(x[n] for n in ARGS), st2, slots=torch.tensor(bad, dtype=torch.int32).cuda(),
                                 check_status=True)
        assert e.value.code == 6
        out = gma.gma_delta_decode(*(x[n] for n in ARGS), states.clone(), slots=torch.tensor(bad, dtype=torch.int32).cuda())
        assert gma.gma_get_status() == 6 and gma.gma_get_status() == 0
        assert not out[1].any() and torch.equal(out[[0, 2, 3]], good[[0, 2, 3]])
        assert torch.equal(st2[[0, 4]], states[[0, 4]]) and torch.equal(st2[[2, 3, 5]], st[[2, 3, 5]])
        assert torch.equal(st2[1], states[1])


@gpu
def test_decode_lengths_and_default_slots(gma):
    x = make(3, 2, 4, 64, 64, seed=17, state=True, lengths=[4, 0, 2])
    want, S = reference(x)
    y = cuda(x)
    st = y["state"].clone()
    out = gma.gma_delta_decode(*(y[n] for n in ARGS), st, lengths=y["lengths"])
    assert off(out, want) <= tol32(4, 64) and off(st, S) <= tol32(4, 64) and torch.equal(st[1], y["state"][1])


@gpu
def test_python_refusals(gma):
    x = cuda(make(2, 4, 8, 64, 64, "bf16", Hk=2))
    a = [x[n] for n in ARGS]
    with pytest.raises(ValueError):
        gma.gma_delta_forward(a[0].transpose(1, 2), *a[1:])
    with pytest.raises(ValueError):
        gma.gma_delta_forward(a[0], a[1].float(), *a[2:])
    with pytest.raises(ValueError):
        gma.gma_delta_forward(*a[:3], a[3][:, :2].contiguous(), a[4])
    with pytest.raises(ValueError):
        gma.gma_delta_forward(*a, lengths=torch.zeros(2, dtype=torch.int64, device="cuda"))
    with pytest.raises(ValueError):
        gma.gma_delta_forward(*a, state=torch.zeros(2, 4, 64, 32, device="cuda"))
    with pytest.raises(ValueError):
        gma.gma_delta_forward(a[0][:, :1].contiguous().expand(-1, 3, -1, -1).contiguous(),
                              a[1][:, :1].expand(-1, 3, -1, -1).contiguous(), *a[2:])
    with pytest.raises(gma.GmaError) as e:
        gma.gma_delta_forward(*a, workspace=torch.zeros(128, dtype=torch.uint8, device="cuda"))
    assert e.value.code == 3
    with pytest.raises(TypeError):
        gma.gma_delta_decode(*a, None)


# ------------------------------------------------------------------------------------------ GPU: offsets past 32 bits

@gpu
def test_sequences_of_more_than_2_31_elements(gma):
    """The last head of a call whose V has more than 2^31 elements, against that head in a call of its own.  The two
    calls may share a head's columns over warps differently: each is within test_forward's and test_backward's bounds."""
    H, N, d, dv = 264, 65536, 64, 128
    assert H * N * dv > 2 ** 31
    gen = torch.Generator("cuda").manual_seed(5)

    def rand(last):
        x = torch.empty((1, H, N, last), dtype=torch.bfloat16, device="cuda")
        return x.normal_(generator=gen)

    def keys():                                          # about unit length
        return rand(d).mul_(d ** -0.5)

    x = [keys(), keys().mul_(0.75), rand(dv), -0.2 * torch.rand((1, H, N), generator=gen, device="cuda"),
         torch.rand((1, H, N), generator=gen, device="cuda")]
    dO = rand(dv)
    out = gma.gma_delta_forward(*x, check_status=True)[:, -1:].clone()
    grads = [t[:, -1:].clone() for t in gma.gma_delta_backward(*x, dO, check_status=True)[:5]]
    one = [t[:, -1:].clone() for t in x]
    dO = dO[:, -1:].clone()
    del x
    near = lambda a, b, lim: float((a.float() - b.float()).abs().max()) <= lim * float(b.float().abs().max())
    try:
        assert near(out, gma.gma_delta_forward(*one), 6 * 2.0 ** -8)
        for a, b in zip(grads, gma.gma_delta_backward(*one, dO)[:5]):
            assert near(a, b, 8 * 2.0 ** -8)
    finally:
        from gaussian_mixture_latent_gb300 import delta
        torch.cuda.synchronize()
        delta._scratch.clear()                           # some tens of GB
        torch.cuda.empty_cache()


@gpu
def test_pools_of_more_than_2_31_elements(gma):
    S, H, d, dv = 2100, 64, 128, 128
    assert (S - 2) * H * d * dv > 2 ** 31
    x = cuda(make(2, H, 1, d, dv, "bf16", seed=8))
    a = [x[n] for n in ARGS]
    pool = torch.empty((S, H, d, dv), device="cuda")
    codes = torch.empty((S, H, d, dv), dtype=torch.int8, device="cuda")
    scales = torch.empty((S, H, d, dv // 32), device="cuda")
    small = torch.randn((2, H, d, dv), device="cuda")
    t = lambda *v: torch.tensor(v, dtype=torch.int32, device="cuda")
    pool[S - 1], pool[3] = small[0], small[1]
    out = gma.gma_delta_decode(*a, pool, slots=t(S - 1, 3), check_status=True)
    assert torch.equal(out, gma.gma_delta_decode(*a, small))
    assert torch.equal(pool[S - 1], small[0]) and torch.equal(pool[3], small[1])
    gma.gma_state_store(pool, codes, scales, src=t(S - 1, 3), dst=t(S - 2, 1), check_status=True)
    gma.gma_state_load(codes, scales, pool, src=t(S - 2, 1), dst=t(S - 2, 0), check_status=True)
    c, s, back = torch.empty_like(codes[:2]), torch.empty_like(scales[:2]), torch.empty_like(small)
    gma.gma_state_store(small, c, s)
    gma.gma_state_load(c, s, back)
    assert torch.equal(codes[S - 2], c[0]) and torch.equal(codes[1], c[1]) and torch.equal(scales[S - 2], s[0])
    assert torch.equal(pool[S - 2], back[0]) and torch.equal(pool[0], back[1])


# ------------------------------------------------------------------------------------------ GPU: streams and graphs

@gpu
def test_two_host_threads_on_one_stream(gma):
    """Calls of several kernels each, from two threads, share the stream's scratch buffer: neither sees the other's."""
    import threading
    xs = [cuda(make(1, 4, n, 64, 64, "bf16", seed=n)) for n in (200, 330)]
    call = lambda x: gma.gma_delta_backward(*(x[n] for n in ARGS), x["dO"])[:5]
    want = [call(x) for x in xs]
    torch.cuda.synchronize()
    wrong, stream = [], torch.cuda.current_stream()

    def work(i):
        with torch.cuda.stream(stream):
            got = [call(xs[i]) for _ in range(200)]
            torch.cuda.synchronize()
            wrong.append(sum(not all(torch.equal(a, b) for a, b in zip(g, want[i])) for g in got))

    threads = [threading.Thread(target=work, args=(i,)) for i in range(2)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert wrong == [0, 0]


@gpu
def test_scale_given_as_a_tensor_is_read_at_each_call(gma):
    x = cuda(make(1, 2, 40, 64, 64, "bf16"))
    a = [x[n] for n in ARGS]
    scale = torch.tensor(0.5)
    first = gma.gma_delta_forward(*a, scale=scale)
    assert torch.equal(first, gma.gma_delta_forward(*a, scale=0.5))
    scale.fill_(0.25)                                    # half of it: a power of two, so that every rounding halves too
    assert torch.equal(gma.gma_delta_forward(*a, scale=scale), first / 2)


@gpu
def test_two_streams_at_once(gma):
    xs = [cuda(make(2, 8, 700, 64, 64, "bf16", seed=s)) for s in (1, 2)]
    want = [gma.gma_delta_backward(*(x[n] for n in ARGS), x["dO"])[:5] for x in xs]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in xs]
    got = [[], []]
    for _ in range(5):
        for i, (x, s) in enumerate(zip(xs, streams)):
            got[i] = gma.gma_delta_backward(*(x[n] for n in ARGS), x["dO"], stream=s)[:5]
    torch.cuda.synchronize()
    for g, w in zip(got, want):
        assert all(torch.equal(a, b) for a, b in zip(g, w))


@gpu
def test_two_graphs_and_an_eager_call_keep_apart(gma):
    xs = [cuda(make(1, 4, 300, 128, 64, "bf16", seed=s, state=True)) for s in (3, 4)]

    def both(x):
        o, S = gma.gma_delta_forward(*(x[n] for n in ARGS), state=x["state"], return_state=True)
        return (o, S) + gma.gma_delta_backward(*(x[n] for n in ARGS), x["dO"], state=x["state"], dstate=x["dstate"])

    want = [both(x) for x in xs]
    torch.cuda.synchronize()
    graphs, outs = [], []
    for x in xs:
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            outs.append(both(x))
        graphs.append(g)
    big = cuda(make(1, 4, 900, 128, 64, "bf16", seed=9))     # a later, larger eager call replaces the eager scratch
    gma.gma_delta_backward(*(big[n] for n in ARGS), big["dO"])
    for t in outs[0] + outs[1]:
        t.zero_()
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        graphs[1].replay()
    graphs[0].replay()
    torch.cuda.synchronize()
    for o, w in zip(outs, want):
        assert all(torch.equal(a, b) for a, b in zip(o, w))


# ------------------------------------------------------------------------------------------ GPU: together

@gpu
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_prefill_park_resume_decode(gma, dtype):
    """A prompt is prefilled, its state parked in the 8-bit cache, read back into two other slots, and decoded on."""
    B, H, Hk, N, d, dv, T = 3, 4, 2, 100, 64, 64, 6
    x = make(B, H, N + T, d, dv, dtype, Hk=Hk, seed=31, lengths=None)
    first = {n: (x[n][:, :, :N] if n in ARGS else x[n]) for n in x}
    rest = {n: (x[n][:, :, N:] if n in ARGS else x[n]) for n in x}
    _, S = reference(first)
    y = cuda(x)
    pool = torch.zeros((8, H, d, dv), device="cuda")
    out, state = gma.gma_delta_forward(*(y[n][:, :, :N].contiguous() for n in ARGS), return_state=True)
    codes = torch.zeros((5, H, d, dv), dtype=torch.int8, device="cuda")
    scales = torch.zeros((5, H, d, (dv + 31) // 32), device="cuda")
    at = torch.tensor([4, 0, 2], dtype=torch.int32, device="cuda")
    gma.gma_state_store(state, codes, scales, dst=at)
    src = torch.tensor([4, 0, 2, 4, 0, 2], dtype=torch.int32, device="cuda")
    dst = torch.tensor([7, 1, 3, 0, 2, 6], dtype=torch.int32, device="cuda")
    gma.gma_state_load(codes, scales, pool, src=src, dst=dst)
    assert not pool[4].any() and not pool[5].any()
    back = pool[dst[:3].long()]
    assert torch.equal(back, pool[dst[3:].long()])
    # the cache is off by half a step of 127 of its group's largest value
    groups = torch.from_numpy(S).reshape(B, H, d, -1, 32).abs().amax(-1, keepdim=True).expand(-1, -1, -1, -1, 32)
    gap = (back.cpu().double() - torch.from_numpy(S)).abs().reshape(groups.shape)
    assert (gap <= groups / 254 + 4 * tol32(N, d) * np.abs(S).max()).all()
    rest["state"] = back.cpu()
    want, after = reference(rest)
    outs = [gma.gma_delta_decode(*(y[n][:, :, N + t:N + t + 1].contiguous() for n in ARGS), pool, slots=dst[:3])
            for t in range(T)]
    lim = tol32(T, d) + (2.0 ** -8 if dtype == "bf16" else 0)
    assert off(torch.cat(outs, 2), want) <= lim and off(pool[dst[:3].long()], after) <= tol32(T, d)
    assert torch.equal(pool[dst[3:].long()], back)
