"""Linear attention with one decay per head on the GPU against its recurrence in float64.

Tolerances, relative to the output's 2-norm (`rel`) unless said otherwise:

* fp32 inputs: every product and sum is fp32 (rounding 2^-24 = 6e-8). A sum of n terms of random sign is off by about
  sqrt(n) 2^-24 of its terms' 2-norm; the longest chains here (128 features, 128 tokens of a chunk, a few hundred decayed
  steps) stay below 2^9 terms: 2^4.5 2^-24 = 1.4e-6. Exponentials of gate sums G carry |G| 2^-24 (|G| <= 32 where they
  matter): 2e-6. Bound: 1e-5.
* bf16 inputs: the output is rounded to bf16 (half a step: 2^-8 of the value, in the 2-norm at most 2^-8, uniformly
  distributed 2^-8 / sqrt(3)), and so are the two operands that the tensor-core path makes itself, the masked scores and
  the state in front of its readout. Three independent errors of rms 2^-8 / sqrt(3) at most: 2^-8. Element by element
  each of the three is at most 2^-8 of the sum of absolute values (`size` of the reference): 3 * 2^-8 of that.
* states are kept in fp32; the operand that enters them on the tensor cores is split in two bf16 parts, 2^-16 at most:
  in the 2-norm 1e-5 as for fp32, element by element 2^-15 of the state of absolute values.
* the gradient of the gates is a sum of fp32 values whose neighbours cancel within one segment (at most 512 tokens); the
  terms left in it have at least 1/sqrt(512) of the 2-norm of what is summed: sqrt(512) 2^-24 8 = 1.1e-5, and for the
  two-part operands (2^-17 at most, rms 2^-19) sqrt(512) 2^-19 = 4.3e-5. Bound: 1e-4.
"""

import numpy as np
import pytest

import head_decay_reference as ref

pytestmark = pytest.mark.gpu

REL = {"f32": 1e-5, "bf16": 2.0 ** -8}


@pytest.fixture(scope="module")
def sdl():
    torch = pytest.importorskip("torch")
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from structured_decay_linear_gb300 import build as nvbuild
    nvbuild.build()
    import structured_decay_linear_gb300 as s
    s.library()
    return s


def rel(a, b):
    a, b = np.asarray(a, np.float64), np.asarray(b, np.float64)
    n = np.linalg.norm(b)
    return float(np.linalg.norm(a - b) / n) if n else float(np.linalg.norm(a))


def host(t):
    return t.detach().double().cpu().numpy()


def make(dtype, B, H, Hq, T, dk, dv, per_head=False, state=True, major=False, rate=0.1, seed=0):
    """Inputs on the device: [B,heads,T,d] views, stored with the tokens first if `major`."""
    import torch
    g = torch.Generator(device="cuda").manual_seed(seed)
    dt = torch.bfloat16 if dtype == "bf16" else torch.float32

    def rows(h, d, scale):
        x = torch.randn((B, T, h, d) if major else (B, h, T, d), device="cuda", generator=g) * scale
        return x.to(dt).transpose(1, 2) if major else x.to(dt)

    x = dict(q=rows(Hq, dk, dk ** -0.5), k=rows(Hq, dk, dk ** -0.5), v=rows(H, dv, 1.0))
    if per_head:
        x["decay"] = -rate * (0.1 + torch.rand(H, device="cuda", generator=g))
    else:
        z = torch.rand((B, T, H) if major else (B, H, T), device="cuda", generator=g)
        x["decay"] = -rate * 2 * (z.transpose(1, 2) if major else z)
    if state:
        x["S0"] = 0.3 * torch.randn(B, H, dk, dv, device="cuda", generator=g)
    return x


def gates(x, shape):
    g = host(x["decay"])
    return np.broadcast_to(g[None, :, None], shape) if g.ndim == 1 else g


def want(x):
    S0 = x.get("S0")
    v = x["v"]
    return ref.forward(host(x["q"]), host(x["k"]), host(v), gates(x, v.shape[:3]), None if S0 is None else host(S0))


def check_forward(dtype, o, S_T, w):
    o_ref, S_ref, size, A = w
    o, S_T = host(o), host(S_T)
    assert np.isfinite(o).all() and np.isfinite(S_T).all()
    assert rel(o, o_ref) <= REL[dtype]
    assert rel(S_T, S_ref) <= REL["f32"]
    step = 3 * 2.0 ** -8 if dtype == "bf16" else 1e-5
    assert (np.abs(o - o_ref) <= step * size + 1e-30).all()
    assert (np.abs(S_T - S_ref) <= 2.0 ** -15 * A + 1e-30).all()


SIZES = [
    # B, H, Hq, T, dk, dv
    (1, 1, 1, 1, 128, 128),
    (2, 3, 3, 2, 64, 64),
    (1, 2, 1, 31, 128, 64),
    (2, 2, 2, 33, 64, 128),
    (1, 4, 2, 127, 128, 128),
    (1, 2, 2, 128, 64, 64),
    (3, 2, 1, 129, 128, 128),
    (1, 3, 3, 300, 128, 64),
    (2, 4, 4, 257, 32, 128),
    (1, 2, 2, 65, 128, 32),
    (1, 2, 2, 200, 32, 32),
    (1, 6, 2, 700, 64, 128),
    (1, 1, 1, 1500, 128, 128),
]


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("B,H,Hq,T,dk,dv", SIZES)
def test_forward(sdl, dtype, B, H, Hq, T, dk, dv):
    x = make(dtype, B, H, Hq, T, dk, dv, per_head=T % 2 == 0, state=T % 3 != 0, major=H % 2 == 0, seed=T)
    f = sdl.HeadDecay(x["q"].dtype, B, H, T, dk, dv, q_heads=Hq, per_head=T % 2 == 0, token_major=T % 4 < 2)
    o, S_T = f(**x)
    assert o.shape == (B, H, T, dv) and o.dtype == x["q"].dtype
    check_forward(dtype, o, S_T, want(x))
    assert f.device_status() == 0
    a, b = o.clone(), S_T.clone()
    o, S_T = f(**x)
    import torch
    assert torch.equal(a, o) and torch.equal(b, S_T)          # the same bits again


@pytest.mark.parametrize("dtype,d", [("f32", 64), ("bf16", 128), ("bf16", 64), ("bf16", 32)])
@pytest.mark.parametrize("kind", ["zero", "forget", "strong", "far"])
def test_gates_at_their_ends(sdl, dtype, d, kind):
    """Gates of 0 (nothing decays), -inf (the state is dropped), strong ones, and sums far below the exponent's range."""
    import torch
    x = make(dtype, 1, 2, 2, 290, d, d, seed=3)
    g = x["decay"]
    if kind == "zero":
        g.zero_()
    elif kind == "forget":
        g[:, 0, [0, 5, 127, 128, 200]] = float("-inf")
        g[:, 1, 289] = float("-inf")
    elif kind == "strong":
        g.mul_(60.0)
    else:
        g.fill_(-1000.0)
        g[:, :, ::2] = -0.01
    f = sdl.HeadDecay(x["q"].dtype, 1, 2, 290, d, d)
    o, S_T = f(**x)
    with np.errstate(all="ignore"):
        check_forward(dtype, o, S_T, want(x))


@pytest.mark.parametrize("dtype,d", [("f32", 64), ("bf16", 128), ("bf16", 32)])
def test_nothing_leaks_between_heads_and_batches(sdl, dtype, d):
    """A batch entry of NaN and infinities leaves the others' results, bit by bit."""
    import torch
    x = make(dtype, 3, 2, 2, 150, d, d, seed=4)
    f = sdl.HeadDecay(x["q"].dtype, 3, 2, 150, d, d)
    o, S = (t.clone() for t in f(**x))
    for name in ("q", "k", "v"):
        x[name][1] = float("nan") if name == "k" else float("inf")
    o2, S2 = f(**x)
    assert torch.equal(o[0::2], o2[0::2]) and torch.equal(S[0::2], S2[0::2])


@pytest.mark.parametrize("dtype,d", [("f32", 64), ("bf16", 128)])
def test_a_sequence_in_two_calls(sdl, dtype, d):
    """S_T of a call continues as S0 of the next, in place too."""
    import torch
    x = make(dtype, 2, 2, 2, 333, d, d, seed=5)
    w = want(x)
    cut = 190
    part = lambda a, b: {n: (t[:, :, a:b] if n != "S0" else t) for n, t in x.items()}  # noqa: E731
    f1, f2 = sdl.HeadDecay(x["q"].dtype, 2, 2, cut, d, d), sdl.HeadDecay(x["q"].dtype, 2, 2, 333 - cut, d, d)
    o1, S1 = f1(**part(0, cut))
    f2.S_T.copy_(S1)
    y = part(cut, 333)
    y["S0"] = f2.S_T                                          # S_T may be S0
    o2, S2 = f2(**y)
    check_forward(dtype, torch.cat([o1, o2], 2), S2, w)


def test_empty_sequence(sdl):
    import torch
    x = make("bf16", 2, 2, 1, 0, 64, 128, seed=6)
    f = sdl.HeadDecay(torch.bfloat16, 2, 2, 0, 64, 128, q_heads=1)
    o, S_T = f(**x)
    assert o.shape == (2, 2, 0, 128) and torch.equal(S_T, x["S0"])
    b = sdl.HeadDecayBackward(torch.bfloat16, 2, 2, 0, 64, 128, q_heads=1)
    dST = torch.randn_like(S_T)
    g = b(torch.empty(2, 2, 0, 128, device="cuda", dtype=torch.bfloat16), dST, **x)
    assert torch.equal(g["S0"], dST)


# ---- gradients

def grads_want(x, dO, dST):
    S0 = x.get("S0")
    v = x["v"]
    w = ref.backward(host(x["q"]), host(x["k"]), host(v), gates(x, v.shape[:3]), host(dO),
                     None if dST is None else host(dST), None if S0 is None else host(S0))
    if x["decay"].dim() == 1:
        w["decay"] = w["decay"].sum((0, 2))
    return w


def check_grads(dtype, got, w):
    for n in w:
        g = host(got[n])
        assert np.isfinite(g).all(), n
        tol = REL["f32"] if n == "S0" else 1e-4 if n == "decay" else REL[dtype]
        assert rel(g, w[n]) <= tol, (n, rel(g, w[n]))


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("B,H,Hq,T,dk,dv", SIZES)
def test_backward(sdl, dtype, B, H, Hq, T, dk, dv):
    import torch
    per_head = T % 2 == 1
    x = make(dtype, B, H, Hq, T, dk, dv, per_head=per_head, state=T % 3 != 1, major=H % 2 == 0, seed=T + 50)
    g = torch.Generator(device="cuda").manual_seed(9)
    dO = torch.randn(B, T, H, dv, device="cuda", generator=g).to(x["q"].dtype).transpose(1, 2)
    dST = 0.3 * torch.randn(B, H, dk, dv, device="cuda", generator=g) if T % 3 != 1 else None
    b = sdl.HeadDecayBackward(x["q"].dtype, B, H, T, dk, dv, q_heads=Hq, per_head=per_head, token_major=T % 4 < 2)
    got = b(dO, dST, **x)
    w = grads_want(x, dO, dST)
    check_grads(dtype, got, w)
    assert b.device_status() == 0
    first = {n: t.clone() for n, t in got.items()}
    got = b(dO, dST, **x)
    assert all(torch.equal(first[n], got[n]) for n in first)
    less = b(dO, dST, **x, decay_grad=False)
    assert "decay" not in less
    if b.path == "hd_fp32":
        assert all(torch.equal(first[n], less[n]) for n in less)
    # on the tensor cores dq and dk then take one-part operands (2^-8, not 2^-16, before the output's own rounding to
    # bf16): not the same bits, but within the bound that counts those roundings
    check_grads(dtype, less, {n: w[n] for n in less})


def test_backward_against_differences(sdl):
    """The gradients of a scalar loss against its differences, f32: the loss's own fp32 noise (1e-7 of |L|) over the
    step leaves 1e-2 of the derivative."""
    import torch
    x = make("f32", 1, 2, 1, 70, 32, 64, seed=11)
    f = sdl.HeadDecay(torch.float32, 1, 2, 70, 32, 64, q_heads=1)
    b = sdl.HeadDecayBackward(torch.float32, 1, 2, 70, 32, 64, q_heads=1)
    dO, dST = torch.randn(1, 2, 70, 64, device="cuda"), torch.randn(1, 2, 32, 64, device="cuda")

    def loss(y):
        o, S = f(**y)
        return float((o.double() * dO.double()).sum() + (S.double() * dST.double()).sum())

    got = {n: t.clone() for n, t in b(dO, dST, **x).items()}
    for n in ("q", "k", "v", "decay", "S0"):
        u = torch.randn_like(x[n])
        h = 1e-2 if n != "decay" else 1e-3
        hi, lo = dict(x), dict(x)
        hi[n], lo[n] = x[n] + h * u, x[n] - h * u
        d = (loss(hi) - loss(lo)) / (2 * h)
        w = float((got[n].double() * u.double()).sum())
        assert abs(d - w) <= 1e-2 * max(abs(w), float(got[n].double().norm())), n


@pytest.mark.parametrize("dtype,d", [("f32", 64), ("bf16", 128)])
def test_backward_with_forgetting_gates(sdl, dtype, d):
    import torch
    x = make(dtype, 1, 2, 2, 290, d, d, seed=13)
    x["decay"][:, 0, [0, 5, 127, 128, 256]] = float("-inf")
    x["decay"][:, 1, 100:200] = -40.0
    dO = torch.randn(1, 2, 290, d, device="cuda").to(x["q"].dtype)
    dST = torch.randn(1, 2, d, d, device="cuda")
    b = sdl.HeadDecayBackward(x["q"].dtype, 1, 2, 290, d, d)
    check_grads(dtype, b(dO, dST, **x), grads_want(x, dO, dST))


# ---- one token at a time

@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("N,H,Hq,dk,dv,slots,per_head", [
    (1, 1, 1, 128, 128, 1, False), (5, 4, 2, 64, 128, 9, True), (7, 2, 2, 32, 32, 8, False), (3, 6, 1, 128, 64, 5, False),
    (300, 2, 2, 32, 128, 310, True), (4, 2, 2, 64, 64, 4, False), (2, 2, 1, 128, 32, 3, True), (2, 2, 1, 64, 32, 3, True),
    (2, 1, 1, 32, 64, 2, False)])
def test_decode(sdl, dtype, N, H, Hq, dk, dv, slots, per_head):
    """Three steps on a pool: rows with a state move it on, idle rows and the other slots stay as they were. One step in
    fp32: o is rounded once (2^-8 for bf16), the state 2^-22."""
    import torch
    g = torch.Generator(device="cuda").manual_seed(N)
    pool = torch.randn(slots, H, dk, dv, device="cuda", generator=g)
    at = torch.randperm(slots, generator=torch.Generator().manual_seed(N))[:N]
    if N > 2:
        at[1] = -1
    slot = at.to("cuda", torch.int32)
    step = sdl.HeadDecayDecode(torch.bfloat16 if dtype == "bf16" else torch.float32, N, H, dk, dv, slots, q_heads=Hq,
                               per_head=per_head)
    S = host(pool).copy()
    live = [i for i in range(N) if at[i] >= 0]
    for t in range(3):
        x = make(dtype, N, H, Hq, 1, dk, dv, per_head=per_head, state=False, seed=100 * N + t)
        o = step(x["q"][:, :, 0], x["k"][:, :, 0], x["v"][:, :, 0], x["decay"] if per_head else x["decay"][:, :, 0], pool,
                 slot)
        part = {n: (y if y.dim() == 1 else y[live]) for n, y in x.items()}
        w_o, w_S, size, _ = ref.forward(host(part["q"]), host(part["k"]), host(part["v"]),
                                        gates(part, (len(live), H, 1)), S[at[live].numpy()])
        S[at[live].numpy()] = w_S
        got = host(o)
        tol = 2.0 ** -8 if dtype == "bf16" else 1e-5
        assert (np.abs(got[live] - w_o[:, :, 0]) <= tol * np.abs(w_o[:, :, 0]) + 1e-5 * size[:, :, 0]).all()
        assert (got[[i for i in range(N) if at[i] < 0]] == 0).all()
    assert np.abs(host(pool) - S).max() <= 1e-5 * np.abs(S).max()
    idle = [s for s in range(slots) if s not in at.tolist()]
    assert (host(pool)[idle] == S[idle]).all()
    assert step.device_status() == 0


def test_decode_bad_rows(sdl):
    """A slot out of range, and a slot that two rows name: the first row has it, the others get zeros and a status."""
    import torch
    x = make("f32", 5, 2, 2, 1, 64, 64, state=False, seed=1)
    a = [x[n][:, :, 0] for n in ("q", "k", "v", "decay")]
    pool = torch.randn(4, 2, 64, 64, device="cuda")
    one, two = pool.clone(), pool.clone()
    step = sdl.HeadDecayDecode(torch.float32, 5, 2, 64, 64, 4)
    good = step(*a, one, torch.tensor([2, -1, -1, 0, -1], device="cuda", dtype=torch.int32)).clone()
    assert step.device_status() == 0
    o = step(*a, two, torch.tensor([2, 4, 2, 0, -7], device="cuda", dtype=torch.int32))
    assert torch.equal(o, good) and torch.equal(one, two)
    assert step.device_status(clear=True) == sdl.dplr.DPLR_ERR_INVALID_ARG and step.device_status() == 0


# ---- ragged batches

def ragged(dtype, lengths, H, Hq, dk, dv, spare, per_head, seed=0):
    n = int(sum(lengths)) + spare
    x = make(dtype, 1, H, Hq, n, dk, dv, per_head=per_head, state=False, major=True, seed=seed)
    return {name: (t if t.dim() == 1 else t[0].transpose(0, 1)) for name, t in x.items()}, n


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("lengths,H,Hq,dk,dv,block,per_head", [
    ([5], 2, 2, 128, 128, 128, False),
    ([128, 0, 1, 129, 300], 2, 1, 128, 64, 128, False),
    ([0, 0, 3], 1, 1, 64, 64, 128, True),
    ([700, 64, 513], 2, 2, 64, 128, 256, True),
    ([33, 31, 32, 65, 1, 1, 1], 3, 3, 32, 32, 32, False),
    ([400, 1, 250], 2, 2, 128, 128, 1024, False),
])
def test_packed(sdl, dtype, lengths, H, Hq, dk, dv, block, per_head):
    """Each request of a ragged batch against its own recurrence; slots of requests without tokens, other slots and rows
    behind the last token stay as they were, whatever the rows hold."""
    import torch
    R, slots = len(lengths), len(lengths) + 3
    x, cap = ragged(dtype, lengths, H, Hq, dk, dv, 37, per_head, seed=sum(lengths))
    for name in ("q", "k", "v"):
        x[name][sum(lengths):] = float("nan")
    pool = torch.randn(slots, H, dk, dv, device="cuda")
    before = host(pool)
    slot = torch.randperm(slots, generator=torch.Generator().manual_seed(1))[:R]
    context = torch.tensor([(0, 7)[r % 2] for r in range(R)])
    plan = sdl.RequestPlan(R, cap, slots, block)
    f = sdl.HeadDecayPacked(x["q"].dtype, R, cap, slots, H, dk, dv, q_heads=Hq, per_head=per_head, plan=plan)
    dev = lambda t: t.to("cuda", torch.int32)  # noqa: E731
    plan(dev(torch.tensor(lengths)), dev(slot), dev(context))
    f.o.fill_(7.0)
    o = f(x["q"], x["k"], x["v"], x["decay"], pool)
    assert plan.device_status() == 0 and f.device_status() == 0
    at = 0
    for r, n in enumerate(lengths):
        s = int(slot[r])
        if n == 0:
            assert (host(pool)[s] == before[s]).all()
            continue
        y = {name: (t if t.dim() == 1 else t[at:at + n].transpose(0, 1)[None]) for name, t in x.items()}
        if context[r] > 0:
            y["S0"] = torch.from_numpy(before[s][None]).float()
        check_forward(dtype, o[at:at + n].transpose(0, 1)[None], pool[s][None], want(y))
        at += n
    assert (host(o)[at:] == 7.0).all()
    idle = [s for s in range(slots) if s not in slot.tolist()]
    assert (host(pool)[idle] == before[idle]).all()


def test_packed_requests_do_not_see_each_other(sdl):
    """A request of NaN and infinities between two others leaves their results, bit by bit."""
    import torch
    lengths = [70, 90, 200]
    for dtype, d in (("bf16", 128), ("f32", 64)):
        x, cap = ragged(dtype, lengths, 2, 2, d, d, 0, False, seed=2)
        call = lambda: sdl.HeadDecayPacked(x["q"].dtype, 3, cap, 3, 2, d, d)  # noqa: E731
        i32 = lambda *v: torch.tensor(v, device="cuda", dtype=torch.int32)  # noqa: E731
        out = []
        for bad in (False, True):
            if bad:
                for name in ("q", "k", "v"):
                    x[name][70:160] = float("inf") if name == "v" else float("nan")
            f = call()
            pool = torch.zeros(3, 2, d, d, device="cuda")
            f.plan(i32(*lengths), i32(0, 1, 2), i32(0, 0, 0))
            out.append((f(x["q"], x["k"], x["v"], x["decay"], pool), pool))
        (o, S), (o2, S2) = out
        assert torch.equal(o[:70], o2[:70]) and torch.equal(o[160:], o2[160:]) and torch.equal(S[0::2], S2[0::2])


@pytest.mark.parametrize("R,longest,cap_extra,slots,block", [
    (1, 1, 0, 1, 32), (3, 40, 5, 3, 64), (600, 9, 100, 700, 128), (1200, 300, 1, 4096, 128), (8192, 3, 0, 1 << 20, 32),
    (5, 0, 0, 5, 128), (4, 0, 77, 9, 64)])
def test_plan(sdl, R, longest, cap_extra, slots, block):
    import torch
    rng = np.random.default_rng(R)
    lengths = rng.integers(0, longest + 1, R)
    slot, context = rng.permutation(slots)[:R], rng.integers(0, 100, R)
    cap = int(lengths.sum()) + cap_extra
    p = sdl.RequestPlan(R, cap, slots, block)
    dev = lambda a: torch.from_numpy(a.astype(np.int32)).to("cuda")  # noqa: E731
    t = p(dev(lengths), dev(slot), dev(context))
    assert p.device_status() == 0
    for name, w in ref.plan(lengths, slot, context, cap, block).items():
        assert np.array_equal(t[name].cpu().numpy(), w), name


@pytest.mark.parametrize("lengths,slots,context", [
    ([3, -1, 2], [0, 1, 2], [0, 0, 0]),
    ([3, 4, 2], [0, 3, 2], [0, 0, 0]),
    ([3, 4, 2], [0, -1, 2], [0, 0, 0]),
    ([3, 4, 2], [0, 2, 2], [0, 0, 0]),
    ([3, 4, 2], [0, 1, 2], [0, -5, 0]),
    ([3, 4, 4], [0, 1, 2], [0, 0, 0]),                        # 11 tokens, capacity 10
    ([2 ** 31 - 1, 2 ** 31 - 1, 2 ** 31 - 1], [0, 1, 2], [0, 0, 0]),
    ([3, 4, 2], [0, 1, 2], [0, 2 ** 31 - 2, 0]),
])
def test_plan_refuses(sdl, lengths, slots, context):
    """Refused lengths: a status, and the tables of a batch without tokens, on which the forward does nothing."""
    import torch
    i32 = lambda v: torch.tensor(v, device="cuda", dtype=torch.int32)  # noqa: E731
    f = sdl.HeadDecayPacked(torch.float32, 3, 10, 3, 1, 32, 32)
    p = f.plan
    t = p(i32(lengths), i32(slots), i32(context))
    assert p.device_status() == sdl.dplr.DPLR_ERR_INVALID_ARG
    assert (t["starts"] == 0).all() and (t["block_starts"] == 0).all()
    assert all((t[n] == -1).all() for n in ("blocks", "token_slot", "token_pos"))
    pool = torch.ones(3, 1, 32, 32, device="cuda")
    x = torch.ones(10, 1, 32, device="cuda")
    o = f(x, x, x, torch.zeros(10, 1, device="cuda"), pool)
    assert (o == 0).all() and (pool == 1).all()
    # zero-length requests may share a slot, or have none
    t = p(i32([3, 0, 0]), i32([1, 1, -9]), i32([0, 0, 0]))
    assert p.device_status() == 0 and int(t["starts"][3]) == 3


def test_serving_run(sdl):
    """A request's prompt in two ragged steps, then single tokens, among other requests: as one recurrence. Outputs are
    rounded to bf16 and the state is carried in fp32, so the forward's tolerance holds throughout."""
    import torch
    H, d, slots = 2, 128, 6
    T = [150, 40, 333]
    total = [t + 4 for t in T]
    x = [make("bf16", 1, H, H, n, d, d, state=False, seed=20 + i) for i, n in enumerate(total)]
    pool = torch.randn(slots, H, d, d, device="cuda")
    slot = torch.tensor([4, 0, 2], device="cuda", dtype=torch.int32)
    outs = [[], [], []]
    done = [0, 0, 0]
    f = sdl.HeadDecayPacked(torch.bfloat16, 3, 400, slots, H, d, d)
    for lengths in ([100, 0, 300], [50, 40, 33]):
        rows = {}
        for name in ("q", "k", "v", "decay"):
            part = [x[r][name][0, :, done[r]:done[r] + n].transpose(0, 1) for r, n in enumerate(lengths)]
            part = torch.cat(part)
            rows[name] = torch.cat([part, part.new_zeros((400 - part.shape[0],) + part.shape[1:])]).contiguous()
        f.plan(torch.tensor(lengths, device="cuda", dtype=torch.int32), slot,
               torch.tensor(done, device="cuda", dtype=torch.int32))
        o = f(rows["q"], rows["k"], rows["v"], rows["decay"], pool)
        at = 0
        for r, n in enumerate(lengths):
            outs[r].append(o[at:at + n].transpose(0, 1).clone())
            at += n
            done[r] += n
    step = sdl.HeadDecayDecode(torch.bfloat16, 3, H, d, d, slots)
    for i in range(4):
        tok = [torch.stack([x[r][name][0, :, T[r] + i] for r in range(3)]) for name in ("q", "k", "v", "decay")]
        o = step(*tok, pool, slot)
        for r in range(3):
            outs[r].append(o[r][:, None].clone())
    for r in range(3):
        check_forward("bf16", torch.cat(outs[r], 1)[None], pool[int(slot[r])][None], want(x[r]))


# ---- streams and graphs

def test_graphs_replay_with_new_inputs_and_lengths(sdl):
    import torch
    i32 = lambda *v: torch.tensor(v, device="cuda", dtype=torch.int32)  # noqa: E731
    d = 128
    x, cap = ragged("bf16", [400], 2, 2, d, d, 0, False, seed=3)
    f = sdl.HeadDecayPacked(torch.bfloat16, 3, cap, 4, 2, d, d, plan=sdl.RequestPlan(3, cap, 4, 128))
    lengths, slot, context = i32(100, 200, 50), i32(3, 1, 0), i32(0, 9, 0)
    pool = torch.randn(4, 2, d, d, device="cuda")
    start = pool.clone()

    def call():
        f.plan(lengths, slot, context)
        return f(x["q"], x["k"], x["v"], x["decay"], pool)

    call()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call()
    for new in ((100, 200, 50), (1, 0, 399), (0, 0, 0), (300, 30, 3)):
        lengths.copy_(i32(*new))
        pool.copy_(start)
        f.o.zero_()
        graph.replay()
        a, b = f.o.clone(), pool.clone()
        pool.copy_(start)
        f.o.zero_()
        o = call()
        assert torch.equal(a, o) and torch.equal(b, pool), new


@pytest.mark.parametrize("dtype,d,T", [("bf16", 128, 700), ("f32", 64, 300)])
def test_forward_and_backward_in_a_graph_and_on_another_stream(sdl, dtype, d, T):
    import torch
    x = make(dtype, 1, 2, 1, T, d, d, seed=8)
    dO = torch.randn(1, 2, T, d, device="cuda").to(x["q"].dtype)
    dST = torch.randn(1, 2, d, d, device="cuda")
    f = sdl.HeadDecay(x["q"].dtype, 1, 2, T, d, d, q_heads=1)
    b = sdl.HeadDecayBackward(x["q"].dtype, 1, 2, T, d, d, q_heads=1)

    def call(stream=None):
        o, S = f(**x, stream=stream)
        g = b(dO, dST, **x, stream=stream)
        return [o, S] + [g[n] for n in sorted(g)]

    first = [t.clone() for t in call()]
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        kept = call()
    for t in kept:
        t.zero_()
    graph.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(a, c) for a, c in zip(first, kept))
    side = torch.cuda.Stream()
    for t in kept:
        t.zero_()
    side.wait_stream(torch.cuda.current_stream())
    other = call(side)
    side.synchronize()
    assert all(torch.equal(a, c) for a, c in zip(first, other))


def test_two_calls_at_once(sdl):
    """Two prepared forwards on two streams: each has its own workspace."""
    import torch
    x, y = (make("bf16", 1, 2, 2, 2000, 128, 128, seed=s) for s in (30, 31))
    f, g = (sdl.HeadDecay(torch.bfloat16, 1, 2, 2000, 128, 128) for _ in range(2))
    wx, wy = [t.clone() for t in f(**x)], [t.clone() for t in g(**y)]
    torch.cuda.synchronize()
    a, b = torch.cuda.Stream(), torch.cuda.Stream()
    for _ in range(5):
        f.o.zero_(), g.o.zero_()
        torch.cuda.synchronize()
        ox, oy = f(**x, stream=a), g(**y, stream=b)
        torch.cuda.synchronize()
        assert all(torch.equal(p, q) for p, q in zip(wx, ox)) and all(torch.equal(p, q) for p, q in zip(wy, oy))


def test_bindings_refuse(sdl):
    import torch
    x = make("bf16", 1, 2, 2, 16, 64, 64, seed=1)
    f = sdl.HeadDecay(torch.bfloat16, 1, 2, 16, 64, 64)
    for name, bad in (("q", x["q"].float()), ("k", x["k"][:, :, :8]), ("v", x["v"].cpu()), ("decay", x["decay"].double()),
                      ("q", x["q"].transpose(2, 3).contiguous().transpose(2, 3)), ("S0", x["S0"].half()),
                      ("v", x["v"][:, :1].expand(1, 2, 16, 64))):
        y = dict(x)
        y[name] = bad
        with pytest.raises(ValueError):
            f(**y)
    with pytest.raises(sdl.DplrError):
        sdl.HeadDecay(torch.bfloat16, 1, 3, 16, 64, 64, q_heads=2)
    with pytest.raises(sdl.DplrError):
        sdl.HeadDecay(torch.bfloat16, 1, 2, 16, 48, 64)
    with pytest.raises(ValueError):
        sdl.HeadDecay(torch.float16, 1, 2, 16, 64, 64)
    p = sdl.HeadDecayPacked(torch.float32, 2, 8, 2, 1, 32, 32)
    z = torch.zeros(8, 1, 32, device="cuda")
    with pytest.raises(ValueError):        # no tables yet
        p(z, z, z, torch.zeros(8, 1, device="cuda"), torch.zeros(2, 1, 32, 32, device="cuda"))


# ---- calls at the edges

@pytest.mark.parametrize("dtype,d", [("f32", 64), ("bf16", 128), ("bf16", 64)])
@pytest.mark.parametrize("T", [100, 700, 1500])
def test_state_in_place(sdl, dtype, d, T):
    """A prepared forward fed with its own S_T: one segment and several give the bits of a call that keeps S0."""
    import torch
    x = make(dtype, 1, 2, 1, T, d, d, seed=40)
    f = sdl.HeadDecay(x["q"].dtype, 1, 2, T, d, d, q_heads=1)
    o, S_T = (t.clone() for t in f(**x))
    for _ in range(3):
        f.S_T.copy_(x["S0"])
        y = dict(x, S0=f.S_T)
        o2, S2 = f(**y)
        assert torch.equal(o, o2) and torch.equal(S_T, S2)


@pytest.mark.parametrize("dtype,d", [("f32", 64), ("bf16", 128), ("bf16", 64)])
def test_rows_on_sixteen_byte_steps(sdl, dtype, d):
    """Rows whose strides are odd multiples of 16 bytes give the bits of contiguous ones, gradients included."""
    import torch
    x = make(dtype, 2, 2, 1, 260, d, d, seed=41)
    dt, pad = x["q"].dtype, 8 if dtype == "bf16" else 4
    dO = torch.randn(2, 2, 260, d, device="cuda").to(dt)
    dST = torch.randn(2, 2, d, d, device="cuda")
    apart = lambda t: torch.full((*t.shape[:-1], d + pad), 7.0, device="cuda", dtype=dt)[..., :d].copy_(t)  # noqa: E731
    y = {n: apart(t) if n in "qkv" else t for n, t in x.items()}
    f = sdl.HeadDecay(dt, 2, 2, 260, d, d, q_heads=1)
    b = sdl.HeadDecayBackward(dt, 2, 2, 260, d, d, q_heads=1)
    first = [t.clone() for t in f(**x)]
    assert all(torch.equal(p, q) for p, q in zip(first, f(**y)))
    grads = {n: t.clone() for n, t in b(dO, dST, **x).items()}
    again = b(apart(dO), dST, **y)
    assert all(torch.equal(grads[n], again[n]) for n in grads)


@pytest.mark.parametrize("dtype,d", [("f32", 64), ("bf16", 128)])
def test_a_gate_that_is_no_number(sdl, dtype, d):
    """A NaN among a head's gates reaches everything behind it and no other head; chunks before it stay as they were."""
    import torch
    x = make(dtype, 1, 3, 3, 700, d, d, seed=42)
    f = sdl.HeadDecay(x["q"].dtype, 1, 3, 700, d, d)
    o, S = (t.clone() for t in f(**x))
    x["decay"][0, 1, 400] = float("nan")
    o2, S2 = f(**x)
    assert torch.equal(o[:, ::2], o2[:, ::2]) and torch.equal(S[:, ::2], S2[:, ::2])
    assert torch.equal(o[0, 1, :384], o2[0, 1, :384])
    assert torch.isnan(o2[0, 1, 400:]).all() and torch.isnan(S2[0, 1]).all()


@pytest.mark.parametrize("B,H,Hq,T,dk,dv", [(3, 2, 1, 129, 128, 128), (1, 6, 2, 700, 64, 128), (2, 2, 2, 513, 128, 64),
                                            (1, 40, 40, 1100, 64, 64), (4, 16, 16, 2048, 128, 128), (2, 32, 16, 2500, 64, 128)])
def test_gradients_give_the_same_bits_every_time(sdl, B, H, Hq, T, dk, dv):
    """Fresh and used workspaces, with the memory between filled with NaN: nothing depends on timing or on what was there."""
    import torch
    x = make("bf16", B, H, Hq, T, dk, dv, seed=43)
    dO = torch.randn(B, H, T, dv, device="cuda").bfloat16()
    dST = torch.randn(B, H, dk, dv, device="cuda")
    first = None
    for _ in range(4):
        junk = [torch.full((1 << 24,), float("nan"), device="cuda") for _ in range(3)]
        del junk
        b = sdl.HeadDecayBackward(torch.bfloat16, B, H, T, dk, dv, q_heads=Hq)
        for _ in range(6):
            got = b(dO, dST, **x)
            first = first or {n: t.clone() for n, t in got.items()}
            assert all(torch.equal(first[n], got[n]) for n in first)
        for _ in range(50):
            b(dO, dST, **x)
        assert all(torch.equal(first[n], b.grads[n]) for n in first) and b.device_status() == 0


@pytest.mark.parametrize("B,H,T,dk,dv", [(1, 16, 16384, 128, 128), (1, 3, 70000, 64, 64), (4, 16, 4096, 128, 64)])
def test_long_forwards_give_the_same_bits_every_time(sdl, B, H, T, dk, dv):
    """Many segments to a CTA, back to back, so that hand-offs between its warps meet in every order: same bits, no wait
    that gives up."""
    import torch
    x = make("bf16", B, H, H, T, dk, dv, seed=50)
    f = sdl.HeadDecay(torch.bfloat16, B, H, T, dk, dv)
    first = [t.clone() for t in f(**x)]
    differ = torch.zeros((), device="cuda", dtype=torch.int64)
    for _ in range(100):
        for a, b in zip(first, f(**x)):
            differ += (a != b).sum()
    assert int(differ) == 0 and f.device_status() == 0


def test_offsets_past_32_bits(sdl):
    """Sequences, and a pool of states, of over 2^31 elements. With gates of -0.5 or less what lies 400 tokens back has
    faded to e^-200, so the last tokens are those of a short sequence."""
    import torch
    H, T, d, tail = 16, 1 << 20, 128, 512
    g = torch.Generator(device="cuda").manual_seed(44)
    rows = lambda: torch.randn(1, T + 300, H, d, device="cuda", generator=g, dtype=torch.bfloat16).transpose(1, 2)  # noqa: E731
    x = dict(q=rows() * d ** -0.5, k=rows() * d ** -0.5, v=rows())
    x["decay"] = -0.5 - torch.rand(1, H, T + 300, device="cuda", generator=g)
    assert x["q"].numel() > 2 ** 31
    f = sdl.HeadDecay(torch.bfloat16, 1, H, T + 300, d, d, token_major=True)
    o, S_T = f(**x)
    heads = slice(14, 16)
    y = {n: t[:, heads, -1024:] for n, t in x.items()}
    o_ref, S_ref, size, A = want(y)
    check_forward("bf16", o[:, heads, -tail:], S_T[:, heads], (o_ref[:, :, -tail:], S_ref, size[:, :, -tail:], A))
    del f, o, S_T, x, y
    slots = 8200
    pool = torch.zeros(slots, H, d, d, device="cuda")
    assert pool.numel() > 2 ** 31
    z = make("bf16", 3, H, H, 1, d, d, seed=45)
    at = torch.tensor([slots - 1, 0, 8191], device="cuda", dtype=torch.int32)
    pool[at.long()] = z["S0"]
    dec = sdl.HeadDecayDecode(torch.bfloat16, 3, H, d, d, slots)
    od = dec(z["q"][:, :, 0], z["k"][:, :, 0], z["v"][:, :, 0], z["decay"][:, :, 0], pool, at)
    check_forward("bf16", od[:, :, None], pool[at.long()], want(z))
    # a request of two segments and one of a single token on the pool's last states
    lengths, n = [600, 1], 601
    w, cap = ragged("bf16", lengths, H, H, d, d, 0, False, seed=46)
    p = sdl.HeadDecayPacked(torch.bfloat16, 2, cap, slots, H, d, d, plan=sdl.RequestPlan(2, cap, slots, 256))
    i32 = lambda *v: torch.tensor(v, device="cuda", dtype=torch.int32)  # noqa: E731
    before = pool[[slots - 1, 8191]].clone()
    p.plan(i32(*lengths), i32(slots - 1, 8191), i32(5, 5))
    op = p(w["q"], w["k"], w["v"], w["decay"], pool)
    for r, (a, b, s) in enumerate(((0, 600, slots - 1), (600, n, 8191))):
        u = {name: t[a:b].transpose(0, 1)[None] for name, t in w.items()}
        u["S0"] = before[r][None]
        check_forward("bf16", op[a:b].transpose(0, 1)[None], pool[s][None], want(u))


def test_many_requests(sdl):
    """As many requests as the tables take, most of one token, each on a state of its own, twice with other lengths."""
    import torch
    R, H, d = 8192, 1, 64
    gen = torch.Generator().manual_seed(47)
    p = sdl.HeadDecayPacked(torch.bfloat16, R, 3 * R, R, H, d, d)
    x, cap = ragged("bf16", [3 * R], H, H, d, d, 0, False, seed=48)
    slot = torch.randperm(R, generator=gen).int()
    zero = torch.zeros(R, dtype=torch.int32, device="cuda")
    for _ in range(2):
        n = torch.randint(0, 4, (R,), generator=gen)
        n[17] = 300
        n = torch.minimum(n, (cap - n.cumsum(0) + n).clamp(min=0))
        pool = torch.zeros(R, H, d, d, device="cuda")
        p.plan(n.int().cuda(), slot.cuda(), zero)
        o = p(x["q"], x["k"], x["v"], x["decay"], pool)
        assert p.plan.device_status() == 0 and p.device_status() == 0
        starts = n.cumsum(0) - n
        for r in (0, 16, 17, 18, 4095, 8190, 8191):
            a, b = int(starts[r]), int(starts[r] + n[r])
            if a == b:
                assert not pool[int(slot[r])].any()
                continue
            u = {name: t[a:b].transpose(0, 1)[None] for name, t in x.items()}
            check_forward("bf16", o[a:b].transpose(0, 1)[None], pool[int(slot[r])][None], want(u))


@pytest.mark.parametrize("what", ["forward", "backward", "packed"])
def test_waits_that_give_up_are_reported(sdl, what):
    """Waits limited to 1000 cycles: the first product of a chunk takes longer, so some wait gives up. The kernels end and
    report it, and with the usual limit the same object is right again."""
    import torch
    T, d = 700, 128
    x = make("bf16", 1, 2, 2, T, d, d, state=False, seed=49)
    if what == "forward":
        f = sdl.HeadDecay(torch.bfloat16, 1, 2, T, d, d)
        call = lambda: dict(zip("oS", f(**x)))  # noqa: E731
    elif what == "backward":
        f = sdl.HeadDecayBackward(torch.bfloat16, 1, 2, T, d, d)
        dO = torch.randn(1, 2, T, d, device="cuda").bfloat16()
        call = lambda: f(dO, None, **x)  # noqa: E731
    else:
        f = sdl.HeadDecayPacked(torch.bfloat16, 2, T, 2, 2, d, d, plan=sdl.RequestPlan(2, T, 2, 256))
        i32 = lambda *v: torch.tensor(v, device="cuda", dtype=torch.int32)  # noqa: E731
        f.plan(i32(600, 100), i32(1, 0), i32(0, 0))
        y = {n: t[0].transpose(0, 1).contiguous() for n, t in x.items()}

        def call():
            pool = torch.zeros(2, 2, d, d, device="cuda")
            return {"o": f(y["q"], y["k"], y["v"], y["decay"], pool), "S": pool}
    first = {n: t.clone() for n, t in call().items()}
    assert f.device_status() == 0
    sdl.dplr_la_set_wait_limit(1000)
    try:
        call()
        torch.cuda.synchronize()
        assert f.device_status(clear=True) == sdl.dplr.DPLR_ERR_TIMEOUT
    finally:
        sdl.dplr_la_set_wait_limit(0)
    got = call()
    assert f.device_status() == 0 and all(torch.equal(first[n], got[n]) for n in first)


@pytest.mark.parametrize("lengths,H,block", [
    ([0] * 60, 8, 128),                                   # more CTAs than blocks: none at all
    ([0] * 30 + [1] + [0] * 30, 4, 2048),
    ([1] * 40 + [900] + [130] * 20 + [0, 0, 2000, 5], 8, 2048),
    ([1] * 40 + [900] + [130] * 20 + [0, 0, 2000, 5], 8, 256),
])
def test_blocks_of_all_lengths(sdl, lengths, H, block):
    """Ragged batches of more blocks than CTAs take at once, which are computed longest first: all requests, and the bits of
    a batch that has each request alone."""
    import torch
    d, R = 64, len(lengths)
    x, cap = ragged("bf16", lengths, H, H, d, d, 40, False, seed=51)
    i32 = lambda v: torch.tensor(v, device="cuda", dtype=torch.int32)  # noqa: E731
    p = sdl.HeadDecayPacked(torch.bfloat16, R, cap, R, H, d, d, plan=sdl.RequestPlan(R, cap, R, block))
    pool = torch.zeros(R, H, d, d, device="cuda")
    p.plan(i32(lengths), i32(list(range(R))), i32([0] * R))
    p.o.fill_(7.0)
    o = p(x["q"], x["k"], x["v"], x["decay"], pool)
    assert p.plan.device_status() == 0 and p.device_status() == 0
    at, seen = 0, set()
    for r, n in enumerate(lengths):
        if n == 0:
            assert not pool[r].any()
        elif n not in seen or n > 100:
            seen.add(n)
            one = sdl.HeadDecayPacked(torch.bfloat16, 1, n, 1, H, d, d, plan=sdl.RequestPlan(1, n, 1, block))
            alone = torch.zeros(1, H, d, d, device="cuda")
            one.plan(i32([n]), i32([0]), i32([0]))
            y = one(*(x[name][at:at + n] for name in ("q", "k", "v", "decay")), alone)
            assert torch.equal(o[at:at + n], y) and torch.equal(pool[r], alone[0])
            u = {name: t[at:at + n].transpose(0, 1)[None] for name, t in x.items()}
            check_forward("bf16", y.transpose(0, 1)[None], alone, want(u))
        at += n
    assert bool((o[at:] == 7.0).all())


@pytest.mark.parametrize("dtype,d,H,block", [("bf16", 128, 2, 2048), ("bf16", 64, 8, 256), ("bf16", 64, 8, 128), ("f32", 64, 2, 128),
                                             ("bf16", 32, 2, 64)])
@pytest.mark.parametrize("bad", ["first", "last", "many", "all"])
def test_slots_that_went_bad_after_planning(sdl, dtype, d, H, block, bad):
    """Slots out of range by the time of the forward: these requests are left out, rows and states as they were, with a
    status; the others' results keep their bits."""
    import torch
    lengths = [300, 5, 0, 700, 128, 1, 33] + [40, 130, 1] * 12 + [513, 2]
    R = len(lengths)
    x, cap = ragged(dtype, lengths, H, H, d, d, 20, False, seed=62)
    i32 = lambda v: torch.tensor(v, device="cuda", dtype=torch.int32)  # noqa: E731
    at = torch.randperm(R, generator=torch.Generator().manual_seed(5)).tolist()
    lost = {"first": [0], "last": [R - 1], "many": [0, 1, 3] + list(range(6, R, 2)), "all": list(range(R))}[bad]
    f = sdl.HeadDecayPacked(x["q"].dtype, R, cap, R, H, d, d, plan=sdl.RequestPlan(R, cap, R, block))
    start = torch.randn(R, H, d, d, device="cuda")
    slot, out = i32(at), []
    f.plan(i32(lengths), slot, i32([r % 2 for r in range(R)]))
    for turn in range(3):
        if turn == 1:
            slot[i32(lost).long()] = i32([(-1, R, 2 ** 31 - 1, -2 ** 31)[i % 4] for i in range(len(lost))])
        elif turn == 2:
            slot.copy_(i32(at))
        pool = start.clone()
        f.o.fill_(7.0)
        f(x["q"], x["k"], x["v"], x["decay"], pool)
        out.append((f.o.clone(), pool))
        assert f.device_status(clear=True) == (sdl.dplr.DPLR_ERR_INVALID_ARG if turn == 1 else 0)
    (o, S), (o2, S2), (o3, S3) = out
    assert torch.equal(o, o3) and torch.equal(S, S3)
    at_row = 0
    for r, n in enumerate(lengths):
        rows = slice(at_row, at_row + n)
        at_row += n
        if r in lost:
            assert (o2[rows] == 7.0).all() and torch.equal(S2[at[r]], start[at[r]])
        else:
            assert torch.equal(o2[rows], o[rows]) and torch.equal(S2[at[r]], S[at[r]])
    assert (o2[at_row:] == 7.0).all()


@pytest.mark.parametrize("block", [1 << 30, (1 << 30) + 32, 2 ** 31 - 32])
def test_blocks_longer_than_anything(sdl, block):
    """A caller's "never split": a length and such a block add up to more than 31 bits. One block a request, and the bits of
    any other block that splits none."""
    import torch
    lengths = [40, 100, 5, 0, 33, 65, 32, 300, 1, 31, 66, 7]
    R, d = len(lengths), 64
    x, cap = ragged("bf16", lengths, 2, 2, d, d, 9, False, seed=64)
    i32 = lambda v: torch.tensor(v, device="cuda", dtype=torch.int32)  # noqa: E731
    out = []
    for b in (2048, block):
        f = sdl.HeadDecayPacked(torch.bfloat16, R, cap, R, 2, d, d, plan=sdl.RequestPlan(R, cap, R, b))
        t = f.plan(i32(lengths), i32(list(range(R))), i32([0] * R))
        assert f.plan.device_status() == 0
        for name, w in ref.plan(lengths, range(R), [0] * R, cap, b).items():
            assert np.array_equal(t[name].cpu().numpy(), w), name
        pool = torch.zeros(R, 2, d, d, device="cuda")
        out.append((f(x["q"], x["k"], x["v"], x["decay"], pool), pool))
        assert f.device_status() == 0
    assert torch.equal(out[0][0], out[1][0]) and torch.equal(out[0][1], out[1][1])


def test_a_block_that_forgets_millions_of_times(sdl):
    """A request of two blocks, the first of 12 million tokens of which each forgets all before it: the sum of the gates
    is past every fixed-point range, and the request ends with its last token alone."""
    import torch
    block, n, d = 12_000_000, 12_000_200, 64
    gen = torch.Generator(device="cuda").manual_seed(61)
    x = torch.empty(n, 1, d, device="cuda", dtype=torch.bfloat16)
    for i in range(0, n, 1_000_000):
        x[i:i + 1_000_000] = torch.randn(min(1_000_000, n - i), 1, d, device="cuda", generator=gen).bfloat16()
    i32 = lambda *v: torch.tensor(v, device="cuda", dtype=torch.int32)  # noqa: E731
    f = sdl.HeadDecayPacked(torch.bfloat16, 1, n, 1, 1, d, d, per_head=True, plan=sdl.RequestPlan(1, n, 1, block))
    pool = torch.randn(1, 1, d, d, device="cuda", generator=gen)
    f.plan(i32(n), i32(0), i32(3))
    o = f(x, x, x, torch.full((1,), float("-inf"), device="cuda"), pool)
    assert f.device_status() == 0
    last = host(x[-1, 0])
    assert rel(host(pool[0, 0]), np.outer(last, last)) <= REL["f32"]
    for a, b in ((0, 300), (block - 300, block + 200)):
        y = host(x[a:b, 0])
        assert rel(host(o[a:b, 0]), (y * y).sum(1, keepdims=True) * y) <= REL["bf16"]


@pytest.mark.parametrize("dtype,d,T", [("bf16", 64, 1 << 21), ("f32", 32, 1 << 22)])
def test_gates_close_to_zero_add_up(sdl, dtype, d, T):
    """A gate of -2^-33.6 a token: nothing for one, 1.7e-4 and 3.3e-4 over a long sequence. Only the first token writes, so
    S_T = e^{gT} S0 + e^{g(T-1)} k_0 v_0^T and o_t = S_t^T q_t without other terms.

    Bound: each of the at most 152 (fp32: 304) segments multiplies a state by one exponential and the last one by one per
    chunk of 128 (32) tokens more, each within 2^-22 of its value and rounded once (2^-24): 7.7e-5 (fp32: 2.2e-4). o adds
    its own error (REL)."""
    import torch
    g = -0.34 * 2.0 ** -32
    dt = torch.bfloat16 if dtype == "bf16" else torch.float32
    gen = torch.Generator(device="cuda").manual_seed(60)
    x = torch.zeros(1, 1, T, d, device="cuda", dtype=dt)
    x[0, 0, 0] = torch.randn(d, device="cuda", generator=gen).to(dt)
    x[0, 0, 1:] = 0
    q = torch.zeros_like(x)
    q[0, 0, -64:] = torch.randn(64, d, device="cuda", generator=gen).to(dt)
    S0 = torch.randn(1, 1, d, d, device="cuda", generator=gen)
    decay = torch.full((1,), g, device="cuda")
    f = sdl.HeadDecay(dt, 1, 1, T, d, d, per_head=True)
    o, S_T = f(q, x, x, decay, S0=S0)
    g = float(decay.double().item())
    w = host(x[0, 0, 0])
    S = np.exp(g * T) * host(S0[0, 0]) + np.exp(g * (T - 1)) * np.outer(w, w)
    segments, chunk = (152, 128) if dtype == "bf16" else (304, 32)
    bound = (segments + T / segments / chunk) * (2.0 ** -22 + 2.0 ** -24)
    assert bound < -g * T                                     # the gates' own effect is larger
    assert rel(host(S_T[0, 0]), S) <= bound
    assert rel(host(o[0, 0, -64:]), host(q[0, 0, -64:]) @ S) <= bound + REL[dtype]
    assert f.device_status() == 0


@pytest.mark.parametrize("lengths,H,Hq,dk,dv,block,per_head", [
    ([33, 31, 32, 65, 1, 0, 200], 3, 3, 128, 128, 32, False),
    ([300, 1, 64, 63, 129], 2, 1, 64, 64, 64, True),
    ([97, 96, 95, 500, 2], 4, 2, 128, 64, 96, False),
    ([400, 161, 7], 2, 2, 64, 128, 160, True),
    ([1, 40] * 30 + [700], 8, 8, 64, 64, 32, False),
    ([130] * 24, 16, 4, 128, 128, 96, False),
])
def test_packed_in_blocks_shorter_than_a_chunk(sdl, lengths, H, Hq, dk, dv, block, per_head):
    """Blocks that are no multiple of 128 tokens put short chunks inside a request on the tensor cores too; each request
    against its own recurrence, twice with the same bits."""
    import torch
    R = len(lengths)
    x, cap = ragged("bf16", lengths, H, Hq, dk, dv, 3, per_head, seed=63)
    for name in ("q", "k", "v"):
        x[name][sum(lengths):] = float("nan")
    i32 = lambda v: torch.tensor(v, device="cuda", dtype=torch.int32)  # noqa: E731
    f = sdl.HeadDecayPacked(torch.bfloat16, R, cap, R, H, dk, dv, q_heads=Hq, per_head=per_head,
                            plan=sdl.RequestPlan(R, cap, R, block))
    assert f.path == "hd_tcgen05"
    start, out = torch.randn(R, H, dk, dv, device="cuda"), []
    f.plan(i32(lengths), i32(list(range(R))), i32([r % 2 for r in range(R)]))
    for _ in range(2):
        pool = start.clone()
        f.o.fill_(7.0)
        f(x["q"], x["k"], x["v"], x["decay"], pool)
        out.append((f.o.clone(), pool))
        assert f.plan.device_status() == 0 and f.device_status() == 0
    (o, pool), (o2, pool2) = out
    assert torch.equal(o, o2) and torch.equal(pool, pool2)
    at = 0
    for r, n in enumerate(lengths):
        if n == 0:
            assert torch.equal(pool[r], start[r])
            continue
        y = {name: (t if t.dim() == 1 else t[at:at + n].transpose(0, 1)[None]) for name, t in x.items()}
        if r % 2:
            y["S0"] = start[r][None]
        check_forward("bf16", o[at:at + n].transpose(0, 1)[None], pool[r][None], want(y))
        at += n
    assert (o[at:] == 7.0).all()


def test_one_object_called_by_several_threads(sdl):
    """A prepared step used by four threads on one stream, each with a pool and inputs of its own: every pool gets its own
    thread's tokens, also if another thread comes between a call's arguments and the C call. (The output is the object's, so
    threads that read it take turns by themselves.)"""
    import threading
    import time

    import torch
    N, H, d, steps, threads = 4, 2, 32, 50, 4
    step = sdl.HeadDecayDecode(torch.float32, N, H, d, d, N)
    launch = step._fn

    def interrupted(*a):
        time.sleep(1e-5)
        return launch(*a)

    slot = torch.arange(N, device="cuda", dtype=torch.int32)
    x = [[make("f32", N, H, H, 1, d, d, state=False, seed=70 + 10 * i + j) for j in range(2)] for i in range(threads)]
    rows = [[[y[n][:, :, 0] for n in ("q", "k", "v", "decay")] for y in xs] for xs in x]
    start = torch.randn(N, H, d, d, device="cuda")

    def run(i, pool):
        for t in range(steps):
            step(*rows[i][t % 2], pool, slot)

    alone = [start.clone() for _ in range(threads)]
    for i in range(threads):
        run(i, alone[i])
    step._fn = interrupted
    for _ in range(3):
        pools = [start.clone() for _ in range(threads)]
        torch.cuda.synchronize()
        team = [threading.Thread(target=run, args=(i, pools[i])) for i in range(threads)]
        for t in team:
            t.start()
        for t in team:
            t.join()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(alone, pools))
