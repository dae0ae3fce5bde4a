"""The elementwise gated recurrence where its arithmetic and its tables have edges: log-gates above 0, values that are not finite in
ragged batches, neighbouring requests without a state."""

import numpy as np
import pytest

import layer_reference as ref
from test_recurrence_gpu import DT, TYPES, dev, f32, near, ragged, sdl  # noqa: F401

pytestmark = pytest.mark.gpu
torch = pytest.importorskip("torch")


# ---- log-gates above 0

# Rounding errors of one token, relative: of a, from the hardware's power of two (2^-22) and from g log2(e) in 32 bits, its
# product and its constant (|g| 2^-23.7); of 1 - a, from the series below |g| = 1/4 (its terms' roundings and what it leaves out,
# 2^-22) or from the difference, which has a's error and a rounding. The scan adds six of 2^-24: its multiply-add and
# product, a warp's and a tile's.
def growing(input, x, g, h0=None, dy=None, dh=None):
    """y, dx, dg, dh0 of log-gates of any sign, each with the bound of its error."""
    B, T, D = x.shape
    a, m = np.exp(g), -np.expm1(g)
    ea = 2.0 ** -22 + np.abs(g) * 2.0 ** -23.7 + 6 * 2.0 ** -24
    one = input == "plain"
    s = np.ones_like(a) if one else m
    es = np.zeros_like(a) if one else np.where(np.abs(g) < 0.25, 2.0 ** -22 * np.abs(m), a * ea) + 2.0 ** -24 * np.abs(m)
    zero = np.zeros((B, D))
    first = zero if h0 is None else h0.astype(np.float64)
    h, M, e = first, np.abs(first), zero
    y, mag, bound = np.empty((B, T, D)), np.empty((B, T, D)), np.empty((B, T, D))
    for t in range(T):
        b = s[:, t] * x[:, t]
        e = a[:, t] * (e + ea[:, t] * M) + es[:, t] * np.abs(x[:, t]) + 2.0 ** -23 * np.abs(b)
        h, M = a[:, t] * h + b, a[:, t] * M + np.abs(b)
        y[:, t], mag[:, t], bound[:, t] = h, M, e
    if dy is None:
        return y, bound
    E = zero if dh is None else dh.astype(np.float64)
    N, eE = np.abs(E), zero
    out = {n: (np.zeros((B, T, D)), np.zeros((B, T, D))) for n in ("x", "gate")}
    for t in range(T - 1, -1, -1):
        hp, Mp, ep = (y[:, t - 1], mag[:, t - 1], bound[:, t - 1]) if t else (first, np.abs(first), zero)
        at, xt = a[:, t], x[:, t]
        Dt, Dm = dy[:, t] + E, np.abs(dy[:, t]) + N
        eD = eE + 2.0 ** -24 * Dm
        out["x"][0][:, t] = s[:, t] * Dt
        out["x"][1][:, t] = np.abs(s[:, t]) * (eD + 2.0 ** -24 * Dm) + es[:, t] * Dm
        through, size = (hp, Mp) if one else (hp - xt, Mp + np.abs(xt))
        out["gate"][0][:, t] = Dt * at * through
        out["gate"][1][:, t] = at * (eD * size + Dm * (ep + (ea[:, t] + 3 * 2.0 ** -24) * size))
        E, N, eE = at * Dt, at * Dm, at * (eD + ea[:, t] * Dm)
    out["h0"] = (E, eE)
    return y, bound, out


def rising(shape, r):
    """Log-gates of which a quarter lie between 0 and 4, at the series' ends among them, and the others forget what those grew."""
    g = -r.uniform(0.5, 2.5, shape)
    up = r.random(shape) < 0.25
    g[up] = r.uniform(0, 4, up.sum())
    g.reshape(-1)[:6] = [0.25, 0.2421875, 0.2578125, 1.0, 2.0, 4.0][:g.size]
    return g


@pytest.mark.parametrize("xt,gt", TYPES)
@pytest.mark.parametrize("input", ["plain", "complement"])
@pytest.mark.parametrize("B,T,D", [(1, 1, 8), (2, 40, 72), (1, 300, 24)])
def test_gates_above_zero(sdl, input, xt, gt, B, T, D):  # noqa: F811
    r = np.random.default_rng(31)
    x, xv = dev(r.standard_normal((B, T, D)), xt)
    g, gv = dev(rising((B, T, D), r), gt)
    dy, dyv = dev(r.standard_normal((B, T, D)), xt)
    h0 = r.standard_normal((B, D)).astype(np.float32)
    f = sdl.GatedRecurrence(DT[xt], B, T, D, "log", input, DT[gt], keep_states=True)
    y, hT = f(x, g, h0=f32(h0))
    want, bound, grads = growing(input, xv, gv, h0, dyv)
    near(y, want, bound, xt, "y")
    near(hT, want[:, -1], bound[:, -1], "f32", "h_T")
    d = sdl.GatedRecurrenceBackward(DT[xt], B, T, D, "log", input, DT[gt])(dy, None, x, g, h0=f32(h0), states=f.states)
    near(d["x"], *grads["x"], xt, "dx")
    near(d["gate"], *grads["gate"], gt, "dgate")
    near(d["h0"], *grads["h0"], "f32", "dh0")


@pytest.mark.parametrize("xt,gt", TYPES)
def test_gates_above_zero_on_a_pool(sdl, xt, gt):  # noqa: F811
    lengths, context, D = [1, 37, 0, 64], [0, 5, 0, 9], 72
    r = np.random.default_rng(32)
    p, x, xv, _, _, S0, slot = ragged(sdl, xt, gt, "log", "complement", lengths, context, D)
    g, gv = dev(rising((sum(lengths), D), r), gt)
    S, at = f32(S0), 0
    y = p(x, g, S)
    for n, s, c in zip(lengths, slot, context):
        if n:
            w, bound = growing("complement", xv[None, at:at + n], gv[None, at:at + n], S0[s:s + 1] if c else None)
            near(y[at:at + n], w[0], bound[0], xt, "y")
            near(S[s], w[0, -1], bound[0, -1], "f32", "state")
        at += n
    N = len(slot)
    S, f = f32(S0), sdl.GatedRecurrenceDecode(DT[xt], N, D, S0.shape[0], "log", "complement", DT[gt])
    y = f(x[:N], g[:N], S, torch.tensor(slot, dtype=torch.int32, device="cuda"))
    for i, s in enumerate(slot):
        w, bound = growing("complement", xv[None, i:i + 1], gv[None, i:i + 1], S0[s:s + 1])
        near(y[i], w[0, 0], bound[0, 0], xt, "one token")
        near(S[s], w[0, 0], bound[0, 0], "f32", "its state")


# ---- what is not finite, in ragged batches

@pytest.mark.parametrize("xt,gt", TYPES)
@pytest.mark.parametrize("gate,value", [("log", -1.0), ("log", -8.0), ("sigmoid", -1.0), ("log", -0.01), ("log", -np.inf)])
def test_packed_not_finite_reaches_what_follows(sdl, gate, value, xt, gt):  # noqa: F811
    """Over tokens and tiles whose product of decays is too small for a number, as the dense forward has it; the request in front, the
    one behind and other channels never see it."""
    lengths, D = [5, 1500, 700], 72
    p, x, xv, g, gv, S0, slot = ragged(sdl, xt, gt, gate, "plain", lengths, [1, 1, 1], D)
    g[...] = value
    S = f32(S0)
    clean, states = p(x, g, S).clone(), S.clone()
    x[8, 3], x[5, 70], x[5 + 600, 40] = float("nan"), float("inf"), float("nan")
    S = f32(S0)
    y = p(x, g, S)
    hit = torch.zeros_like(y, dtype=torch.bool)
    hit[8:1505, 3] = hit[5:1505, 70] = hit[605:1505, 40] = True
    assert torch.equal(y[~hit], clean[~hit]) and not torch.isfinite(y[hit]).any()
    bad = torch.zeros_like(S, dtype=torch.bool)
    bad[slot[1], [3, 40, 70]] = True
    assert torch.equal(S[~bad], states[~bad]) and not torch.isfinite(S[bad]).any()
    dense = sdl.GatedRecurrence(DT[xt], 1, 1500, D, gate, "plain", DT[gt])
    h0 = f32(S0[slot[1]:slot[1] + 1])
    yd, hd = dense(x[None, 5:1505], g[None, 5:1505], h0=h0)
    assert torch.equal(torch.isfinite(yd[0]), torch.isfinite(y[5:1505]))
    assert torch.equal(torch.isfinite(hd[0]), torch.isfinite(S[slot[1]]))


@pytest.mark.parametrize("gate", ["log", "sigmoid"])
def test_decays_are_not_below_zero(sdl, gate):  # noqa: F811
    """A start in a ragged batch is told by a factor of -0, so no gate may give one: a state of 1 without an input becomes a."""
    g = torch.cat([torch.linspace(-110, -80, 20000), torch.linspace(-1000, 0, 20001), torch.tensor([-float("inf"), -3e38, -88.0])])
    D = g.numel()
    f = sdl.GatedRecurrenceDecode(torch.float32, 1, D, 1, gate, "plain")
    wide = torch.zeros(1, D + -D % 4, device="cuda")
    wide[0, :D] = g.cuda()
    S = torch.ones(1, D, device="cuda")
    f(torch.zeros_like(wide)[:, :D], wide[:, :D], S, torch.zeros(1, dtype=torch.int32, device="cuda"))
    assert not torch.signbit(S).any() and (S[0, -3:-1] == 0).all()


# ---- requests without a state beside one another

@pytest.mark.parametrize("xt,gt", TYPES)
@pytest.mark.parametrize("bad", [-1, 1 << 19])
@pytest.mark.parametrize("lengths", [[30, 40, 50], [300, 1, 2, 400, 0, 17]])
def test_neighbours_without_a_state(sdl, xt, gt, bad, lengths):  # noqa: F811
    """Rows whose slots have become the same number out of range: each of their requests starts from zero and leaves no state, also
    where its positions go on where the request in front ends."""
    D = 72
    context = [7 if i == 0 else 7 + sum(lengths[:i]) for i in range(len(lengths))]
    p, x, xv, g, gv, S0, slot = ragged(sdl, xt, gt, "log", "plain", lengths, context, D)
    last = sum(lengths[:-1])
    p.plan.token_slot[:last] = bad
    S = f32(S0)
    y = p(x, g, S)
    assert p.device_status(clear=True) == sdl.dplr.DPLR_ERR_INVALID_ARG
    at = 0
    for i, n in enumerate(lengths):
        if n:
            h0 = S0[slot[i]:slot[i] + 1] if at >= last else None
            w, bound, _ = ref.recurrence("log", "plain", xv[None, at:at + n], gv[None, at:at + n], h0)
            near(y[at:at + n], w[0], bound[0], xt, f"request {i}")
        at += n
    near(S[slot[-1]], w[0, -1], bound[0, -1], "f32", "state")
    others = [i for i in range(S0.shape[0]) if i != slot[-1]]
    assert torch.equal(S[others], f32(S0)[others])
