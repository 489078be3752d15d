"""The gated delta rule and the quantised state cache: cases to measure, their plain forms and their exact values.

Operators (``op`` of a case):
  forward   gma_delta_forward: a whole sequence in chunks, with or without a carried state
  backward  gma_delta_backward: its gradient
  decode    gma_delta_decode: the next token, or a few, of many sequences whose states lie in a pool of slots
  park      gma_state_store, then gma_state_load: states put away in 8 bits and read back
  resume    gma_state_load: states read back from an 8-bit cache into a pool

Per head:  w_t = v_t - e^{g_t} S_{t-1}^T k_t,  S_t = e^{g_t} S_{t-1} + k_t (beta_t w_t)^T,  o_t = scale S_t^T q_t.
"""
import math

import torch

own = False

CHUNK = 64
RESET = -1.0e4          # a log decay that forgets everything: a document boundary in a packed sequence
_DT = {"bf16": torch.bfloat16, "f32": torch.float32}


def _seq(name, op, B, H, N, d, dv, dtype, gates, Hk=None, state=False, ragged=False, resets=False):
    c = dict(op=op, B=B, H=H, Hk=Hk or H, N=N, d=d, dv=dv, dtype=dtype, gates=gates, state=state, ragged=ragged,
             resets=resets)
    return dict(c, name=name) if name else c


def _dec(name, B, H, N, d, dv, dtype, pool, Hk=None):
    c = dict(op="decode", B=B, H=H, Hk=Hk or H, N=N, d=d, dv=dv, dtype=dtype, gates="f32", pool=pool)
    return dict(c, name=name) if name else c


def _cache(name, op, n, H, rows, cols, pool, shared=False):
    c = dict(op=op, n=n, H=H, rows=rows, cols=cols, pool=pool, shared=shared)
    return dict(c, name=name) if name else c


def listed():
    return [
        # a short turn appended to a chat: 45 tokens onto a state that the server holds
        _seq("forward_turn", "forward", 1, 16, 45, 128, 128, "bf16", "f32", Hk=8, state=True),
        # a training step's forward at the library's benchmark shape (8 x 12 heads, 8192 rows, width 64)
        _seq("forward_train", "forward", 8, 12, 8192, 64, 64, "bf16", "bf16"),
        # prefill of one long prompt: the whole state comes back for the decode that follows
        _seq("forward_long", "forward", 1, 32, 32768, 128, 128, "bf16", "f32", Hk=16, state=True),
        # a padded batch of prompts of different lengths, float32, packed documents
        _seq("forward_ragged_f32", "forward", 5, 6, 1531, 64, 64, "f32", "f32", state=True, ragged=True, resets=True),
        # the gradient of the training step above
        _seq("backward_train", "backward", 8, 12, 8192, 64, 64, "bf16", "bf16"),
        # a smaller batch of wider heads, two value heads to a key head, padded
        _seq("backward_shared", "backward", 2, 8, 1999, 128, 128, "bf16", "bf16", Hk=4, ragged=True),
        # float32 training of a small model in segments: the state's gradient goes to the segment before
        _seq("backward_f32", "backward", 2, 4, 515, 64, 128, "f32", "f32", state=True, resets=True),
        # one token of one sequence: latency
        _dec("decode_one", 1, 12, 1, 64, 64, "bf16", 4),
        # one token of each of 256 sequences in a server's pool
        _dec("decode_batch", 256, 32, 1, 128, 128, "bf16", 300, Hk=16),
        # one idle session's mixture memories ([K, dv + 1] per head) put away and read back
        _cache("park_one", "park", 1, 12, 64, 65, 4),
        # 96 sessions of wide heads put away and read back
        _cache("park_batch", "park", 96, 32, 128, 128, 128),
        # one cached prefix read into the slots of 64 new requests
        _cache("resume_prefix", "resume", 64, 32, 128, 128, 100, shared=True),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 1)))))))


def draw(rng):
    op = rng.choice(["forward", "forward", "backward", "backward", "decode", "park", "resume"])
    if op in ("forward", "backward"):
        dtype = rng.choice(["bf16", "bf16", "bf16", "f32"])
        H, ratio = rng.choice([4, 8, 12, 16, 32]), rng.choice([1, 1, 2, 4])
        B = _log(rng, 1, 8)
        d, dv = rng.choice([64, 64, 128, 128, 32, 96]), rng.choice([64, 64, 128, 128, 48, 80])
        most = {"forward": 1 << 19, "backward": 1 << 18}[op] >> (2 if dtype == "f32" else 0)
        N = _log(rng, 1, min(16384, max(1, most // (B * H))))
        return _seq(None, op, B, H, N, d, dv, dtype, "f32" if dtype == "f32" else "bf16" if op == "backward" else
                    rng.choice(["f32", "bf16"]), Hk=H // ratio, state=rng.random() < 0.5 and
                    (op == "forward" or dtype == "f32"), ragged=rng.random() < 0.5, resets=rng.random() < 0.3)
    H = rng.choice([4, 8, 12, 16, 32])
    if op == "decode":
        B, ratio = _log(rng, 1, 200), rng.choice([1, 1, 2, 4])
        return _dec(None, B, H, rng.choice([1, 1, 1, 2, 3, 5]), rng.choice([64, 128, 128, 96]),
                    rng.choice([64, 128, 128, 80]), rng.choice(["bf16", "bf16", "f32"]), B + rng.randrange(1, 40),
                    Hk=H // ratio)
    n = _log(rng, 1, 90)
    return _cache(None, op, n, H, rng.choice([64, 128, 96]), rng.choice([64, 65, 128, 129, 80]),
                  n + rng.randrange(0, 30), shared=op == "resume" and rng.random() < 0.5)


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)

    def normal(*shape):
        return torch.randn(shape, generator=gen, device="cuda")

    if case["op"] in ("park", "resume"):
        n, pool = case["n"], case["pool"]
        shape = (pool, case["H"], case["rows"], case["cols"])
        groups = shape[:3] + ((case["cols"] + 31) // 32,)
        src = torch.randperm(pool, generator=gen, device="cuda")[:n].to(torch.int32)
        if case["shared"]:
            src = src[:1].expand(n).contiguous()
        dst = torch.randperm(pool, generator=gen, device="cuda")[:n].to(torch.int32)
        s = dict(case=case, src=src, dst=dst, codes=torch.zeros(shape, dtype=torch.int8, device="cuda"),
                 scales=torch.zeros(groups, device="cuda"))
        if case["op"] == "park":
            # row magnitudes differ as those of a real state's key directions do
            s["state"] = normal(*shape) * torch.exp(1.5 * normal(*shape[:3], 1))
            s["back"] = torch.zeros(shape, device="cuda")
        else:
            s["codes"] = (40.0 * normal(*shape)).round().clamp(-127, 127).to(torch.int8)
            s["scales"] = torch.exp(normal(*groups) - 4.0)
            s["back"] = torch.zeros(shape, device="cuda")
        return s

    B, H, Hk, N, d, dv = (case[x] for x in ("B", "H", "Hk", "N", "d", "dv"))
    dt, gt = _DT[case["dtype"]], _DT[case["gates"]]

    def unit(x):
        return x / x.norm(dim=-1, keepdim=True)

    # unit routing vectors with a common part, so that keys repeat themselves as those of text do
    common = normal(B, Hk, 1, d)
    q = unit(normal(B, Hk, N, d) + 0.3 * common).to(dt)
    k = unit(normal(B, Hk, N, d) + 0.5 * common).to(dt)
    v = normal(B, H, N, dv).to(dt)
    # per-head decay rates from about 1e-3 to about 1 a token
    rate = torch.exp(torch.linspace(-6.0, 0.5, H, device="cuda"))[:, None]
    g = (-rate * torch.nn.functional.softplus(normal(B, H, N))).to(gt)
    if case.get("resets"):
        g = torch.where(torch.rand((B, 1, N), generator=gen, device="cuda") < 0.01, RESET, g).to(gt)
    beta = torch.sigmoid(normal(B, H, N)).to(gt)
    s = dict(case=case, q=q, k=k, v=v, g=g, beta=beta, state=None, dstate=None, lengths=None)
    if case.get("ragged"):
        u = torch.rand((B,), generator=gen, device="cuda")
        s["lengths"] = (u * (N + 1)).to(torch.int32).clamp(max=N)
        s["lengths"][0] = N
        dead = torch.arange(N, device="cuda")[None] >= s["lengths"][:, None]
        for x in (q, k, v):
            x.masked_fill_(dead[:, None, :, None], float("nan"))   # what padding holds is nobody's business
    if case["op"] == "decode":
        s["state"] = 0.3 * normal(case["pool"], H, d, dv)
        s["slots"] = torch.randperm(case["pool"], generator=gen, device="cuda")[:B].to(torch.int32)
    elif case["state"]:
        s["state"] = 0.3 * normal(B, H, d, dv)
        if case["op"] == "backward":
            s["dstate"] = 0.3 * normal(B, H, d, dv)
    if case["op"] == "backward":
        s["dout"] = normal(B, H, N, dv).to(dt)
        if s["lengths"] is not None:
            s["dout"].masked_fill_(dead[:, None, :, None], float("nan"))
    return s


# ---------------------------------------------------------------------------- plain forms (32 bits)

def _live(s, x):
    """x with zeros in the rows at and past each sequence's length."""
    if s["lengths"] is None:
        return x
    dead = torch.arange(x.shape[2], device=x.device)[None] >= s["lengths"][:, None]
    return x.masked_fill(dead[:, None, :, None] if x.dim() == 4 else dead[:, None], 0.0)


def _wide(s, dtype):
    """q, k, v, g, beta of every value head in `dtype`, padding zeroed."""
    r = s["case"]["H"] // s["case"]["Hk"]
    q, k = (_live(s, s[x]).to(dtype).repeat_interleave(r, dim=1) for x in ("q", "k"))
    return (q, k) + tuple(_live(s, s[x]).to(dtype) for x in ("v", "g", "beta"))


def _plain_inverse(A):
    """(I + A)^-1 of strictly lower triangular A [..., C, C], row by row."""
    C = A.shape[-1]
    T = torch.eye(C, device=A.device, dtype=A.dtype).expand(A.shape).contiguous()
    for i in range(1, C):
        T[..., i, :i] = -(A[..., i:i + 1, :i] @ T[..., :i, :i])[..., 0, :]
    return T


def _plain_delta(q, k, v, g, beta, state, scale):
    """(out, state after the last row) in 32 bits, in chunks; differentiable."""
    B, H, N, d = q.shape
    dv, C = v.shape[-1], CHUNK
    pad = -N % C
    if pad:
        q, k, v = (torch.nn.functional.pad(x, (0, 0, 0, pad)) for x in (q, k, v))
        g, beta = (torch.nn.functional.pad(x, (0, pad)) for x in (g, beta))
    nc = (N + pad) // C
    q, k, v = (x.reshape(B, H, nc, C, x.shape[-1]) for x in (q, k, v))
    beta = beta.reshape(B, H, nc, C, 1)
    G = g.double().reshape(B, H, nc, C).cumsum(-1)     # differences of long sums: 64 bits
    rows = torch.arange(C, device=q.device)
    gap = (G[..., :, None] - G[..., None, :]).masked_fill(rows[:, None] < rows[None], -math.inf)
    D = gap.float().exp()
    e, last = G.float().exp()[..., None], G[..., -1:].float().exp()[..., None]
    f = (G[..., -1:] - G).float().exp()[..., None]
    A = (beta * D * (k @ k.transpose(-1, -2))).masked_fill(rows[:, None] <= rows[None], 0.0)
    with torch.no_grad():
        T = _plain_inverse(A.detach())
    if A.requires_grad:                                # the same values, with the inverse's derivative
        T = T @ (2 * torch.eye(C, device=q.device) - T - A @ T)
    P = D * (q @ k.transpose(-1, -2))
    S = torch.zeros((B, H, d, dv), device=q.device) if state is None else state
    outs = []
    for c in range(nc):
        kc = k[:, :, c]
        u = T[:, :, c] @ (beta[:, :, c] * (v[:, :, c] - e[:, :, c] * (kc @ S)))
        outs.append(e[:, :, c] * (q[:, :, c] @ S) + P[:, :, c] @ u)
        S = last[:, :, c] * S + (f[:, :, c] * kc).transpose(-1, -2) @ u
    out = scale * torch.stack(outs, 2).reshape(B, H, nc * C, dv)[:, :, :N]
    return out, S


def _plain_forward(s):
    q, k, v, g, beta = _wide(s, torch.float32)
    out, S = _plain_delta(q, k, v, g, beta, s["state"], s["case"]["d"] ** -0.5)
    out = _live(s, out).to(s["v"].dtype)
    return {"out": out, "state": S} if s["case"]["state"] else {"out": out}


def _plain_backward(s):
    leaf = {x: _live(s, s[x]).float().requires_grad_() for x in ("q", "k", "v", "g", "beta")}
    if s["state"] is not None:
        leaf["state"] = s["state"].clone().requires_grad_()
    r = s["case"]["H"] // s["case"]["Hk"]
    out, S = _plain_delta(leaf["q"].repeat_interleave(r, dim=1), leaf["k"].repeat_interleave(r, dim=1), leaf["v"],
                          leaf["g"], leaf["beta"], leaf.get("state"), s["case"]["d"] ** -0.5)
    ends, into = [out], [_live(s, s["dout"]).float()]
    if s["dstate"] is not None:
        ends, into = ends + [S], into + [s["dstate"]]
    grads = torch.autograd.grad(ends, list(leaf.values()), into)
    return {"d" + x: _live(s, dx).to(s[x].dtype) if x != "state" else dx for x, dx in zip(leaf, grads)}


def _plain_decode(s):
    q, k, v, g, beta = _wide(s, torch.float32)
    slots = s["slots"].long()
    S = s["state"][slots]
    outs = []
    for t in range(q.shape[2]):
        kt = k[:, :, t, :, None]
        S = g[:, :, t].exp()[..., None, None] * S
        u = beta[:, :, t, None] * (v[:, :, t] - (S * kt).sum(-2))
        S = S + kt * u[:, :, None]
        outs.append((S * q[:, :, t, :, None]).sum(-2))
    s["state"][slots] = S
    return {"out": (s["case"]["d"] ** -0.5 * torch.stack(outs, 2)).to(s["v"].dtype), "state": s["state"]}


def _grouped(x):
    """The last axis in groups of 32, zeros after its end."""
    return torch.nn.functional.pad(x, (0, -x.shape[-1] % 32)).reshape(x.shape[:-1] + (-1, 32))


def _plain_load(s):
    kept, to = ("src", "dst") if s["case"]["op"] == "resume" else ("dst", "src")
    codes, scales = s["codes"][s[kept].long()], s["scales"][s[kept].long()]
    s["back"][s[to].long()] = (_grouped(codes.float()) * scales[..., None]).flatten(-2)[..., :s["case"]["cols"]]
    return {"back": s["back"]}


def _plain_park(s):
    x = _grouped(s["state"][s["src"].long()])
    scale = x.abs().amax(-1) / 127.0
    codes = torch.where(scale[..., None] > 0, x / scale[..., None], torch.zeros_like(x)).round().clamp(-127, 127)
    s["codes"][s["dst"].long()] = codes.flatten(-2)[..., :s["case"]["cols"]].to(torch.int8)
    s["scales"][s["dst"].long()] = scale
    return _plain_load(s)


# ---------------------------------------------------------------------------- one pass

def run(state):
    s = state
    op = s["case"]["op"]
    if not own:
        return {"forward": _plain_forward, "backward": _plain_backward, "decode": _plain_decode, "park": _plain_park,
                "resume": _plain_load}[op](s)
    import gaussian_mixture_latent_gb300 as gma
    if op == "forward":
        r = gma.gma_delta_forward(s["q"], s["k"], s["v"], s["g"], s["beta"], state=s["state"], lengths=s["lengths"],
                                  return_state=s["case"]["state"])
        return {"out": r[0], "state": r[1]} if s["case"]["state"] else {"out": r}
    if op == "backward":
        dq, dk, dv, dg, dbeta, dstate = gma.gma_delta_backward(
            s["q"], s["k"], s["v"], s["g"], s["beta"], s["dout"], state=s["state"], dstate=s["dstate"],
            lengths=s["lengths"])
        r = {"dq": dq, "dk": dk, "dv": dv, "dg": dg, "dbeta": dbeta}
        return dict(r, dstate=dstate) if s["state"] is not None else r
    if op == "decode":
        out = gma.gma_delta_decode(s["q"], s["k"], s["v"], s["g"], s["beta"], s["state"], slots=s["slots"])
        return {"out": out, "state": s["state"]}
    if op == "park":
        gma.gma_state_store(s["state"], s["codes"], s["scales"], src=s["src"], dst=s["dst"])
        gma.gma_state_load(s["codes"], s["scales"], s["back"], src=s["dst"], dst=s["src"])
    else:
        gma.gma_state_load(s["codes"], s["scales"], s["back"], src=s["src"], dst=s["dst"])
    return {"back": s["back"]}


# ---------------------------------------------------------------------------- least work

def work(case):
    """Each input read once and each output written once; products of the recurrence (three [d x dv] products a row
    forward, nine backward: the states again, the reverse recurrence and the gradients)."""
    if case["op"] in ("park", "resume"):
        one = case["H"] * case["rows"] * case["cols"]
        packed = case["H"] * case["rows"] * (case["cols"] + 4 * ((case["cols"] + 31) // 32))
        n = case["n"]
        if case["op"] == "park":
            return {"bytes": n * (8 * one + 2 * packed), "flops": 3 * n * one}
        return {"bytes": n * 4 * one + (1 if case["shared"] else n) * packed, "flops": n * one}
    B, H, Hk, N, d, dv = (case[x] for x in ("B", "H", "Hk", "N", "d", "dv"))
    e, ge = (2 if case["dtype"] == "bf16" else 4), (2 if case["gates"] == "bf16" else 4)
    rows = B * N * (0.5 * (1 + 1 / B) if case.get("ragged") else 1.0)   # one sequence is whole, the others half on average
    ins = 2 * Hk * d * e + H * (dv * e + 2 * ge)
    S = 4 * B * H * d * dv
    if case["op"] == "forward":
        return {"bytes": rows * (ins + H * dv * e) + (2 * S if case["state"] else 0), "flops": rows * H * 6 * d * dv}
    if case["op"] == "backward":
        return {"bytes": rows * (2 * ins + H * dv * e) + (3 * S if case["state"] else 0),
                "flops": rows * H * 18 * d * dv}
    return {"bytes": rows * (ins + H * dv * e) + 2 * S, "flops": rows * H * 6 * d * dv}


# ---------------------------------------------------------------------------- exact values (64 bits, row by row)

def _outer(a, b):
    return a.unsqueeze(-1) * b.unsqueeze(-2)


def _exact_rows(s):
    """The inputs in 64 bits by row: q, k [N, B, H, d], v [N, B, H, dv], decay, beta [N, B, H]."""
    q, k, v, g, beta = _wide(s, torch.float64)
    return [x.movedim(2, 0).contiguous() for x in (q, k, v, g.exp(), beta)]


def _exact_step(S, k, v, a, beta):
    S = a[..., None, None] * S
    w = v - torch.matmul(k.unsqueeze(-2), S).squeeze(-2)
    return S, w, S + _outer(k, beta[..., None] * w)


def _exact_start(s):
    c = s["case"]
    zero = torch.zeros((c["B"], c["H"], c["d"], c["dv"]), dtype=torch.float64, device="cuda")
    if c["op"] == "decode":
        return s["state"][s["slots"].long()].double()
    return zero if s["state"] is None else s["state"].double()


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] in ("park", "resume"):
        # the format fixes the scale and the quotient as 32-bit values; the rest is in 64 bits
        back = s["back"].double()
        for i in range(case["n"]):
            a, b = int(s["src"][i]), int(s["dst"][i])
            if case["op"] == "park":
                x = _grouped(s["state"][a].double())
                scale = (x.abs().amax(-1) / 127.0).float().double()[..., None]
                codes = torch.where(scale > 0, (x / scale).float().double(), 0.0).round()
                back[a] = (codes * scale).flatten(-2)[..., :case["cols"]]
            else:
                x = _grouped(s["codes"][a].double()) * s["scales"][a].double()[..., None]
                back[b] = x.flatten(-2)[..., :case["cols"]]
        return {"back": back}
    q, k, v, a, beta = _exact_rows(s)
    N, scale = q.shape[0], case["d"] ** -0.5
    S = _exact_start(s)
    if case["op"] != "backward":
        out = torch.empty(v.shape, dtype=torch.float64, device="cuda")
        for t in range(N):
            S = _exact_step(S, k[t], v[t], a[t], beta[t])[2]
            out[t] = scale * torch.matmul(q[t].unsqueeze(-2), S).squeeze(-2)
        out = _live(s, out.movedim(0, 2))
        if case["op"] == "decode":
            pool = s["state"].double()
            pool[s["slots"].long()] = S
            return {"out": out, "state": pool}
        return {"out": out, "state": S} if case["state"] else {"out": out}
    # the states at every 64th row, then the rows again from the last block to the first
    starts = []
    for t in range(N):
        if t % 64 == 0:
            starts.append(S)
        S = _exact_step(S, k[t], v[t], a[t], beta[t])[2]
    do = _live(s, s["dout"]).double().movedim(2, 0)
    dS = torch.zeros_like(S) if s["dstate"] is None else s["dstate"].double()
    dq, dk, dv, da, db = (torch.zeros_like(x) for x in (q, k, v, a, beta))
    for first in range((N - 1) // 64 * 64, -1, -64):
        S, kept = starts[first // 64], []
        for t in range(first, min(N, first + 64)):
            kept.append(_exact_step(S, k[t], v[t], a[t], beta[t]) + (S,))
            S = kept[-1][2]
        for t in range(min(N, first + 64) - 1, first - 1, -1):
            faded, w, after, before = kept[t - first]
            dq[t] = scale * (after * do[t].unsqueeze(-2)).sum(-1)
            dS = dS + scale * _outer(q[t], do[t])
            u, du = beta[t][..., None] * w, torch.matmul(k[t].unsqueeze(-2), dS).squeeze(-2)
            db[t], dv[t] = (du * w).sum(-1), beta[t][..., None] * du
            dk[t] = (dS * u.unsqueeze(-2)).sum(-1) - (faded * dv[t].unsqueeze(-2)).sum(-1)
            dS = dS - _outer(k[t], dv[t])
            da[t] = (dS * before).sum((-1, -2))
            dS = a[t][..., None, None] * dS
    r = case["H"] // case["Hk"]

    def keys(x):
        x = x.movedim(0, 2)
        return _live(s, x.reshape(x.shape[0], case["Hk"], r, N, x.shape[-1]).sum(2))

    got = {"dq": keys(dq), "dk": keys(dk), "dv": _live(s, dv.movedim(0, 2)),
           "dg": _live(s, (da * a).movedim(0, 2)), "dbeta": _live(s, db.movedim(0, 2))}
    return dict(got, dstate=dS) if s["state"] is not None else got
