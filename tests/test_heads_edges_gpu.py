"""Head norms and rotary positions where they have edges: rows without a token in an object that is called again, values that are not
finite beside the rotated part, the angles' own precision."""

import numpy as np
import pytest

import layer_reference as ref
from test_heads_gpu import BASE, make, values, weights
from test_recurrence_gpu import DT, dev, near, sdl  # noqa: F401

pytestmark = pytest.mark.gpu
torch = pytest.importorskip("torch")


# ---- rows without a token

@pytest.mark.parametrize("t,gt", [("bf16", "bf16"), ("bf16", "f32"), ("f32", "f32")])
@pytest.mark.parametrize("norm,weighted", [(None, False), ("rms", True), ("l2", False)])
@pytest.mark.parametrize("B,T,Hq,Hk,d,rot", [(2, 7, 3, 1, 64, 16), (9, 1, 5, 0, 256, 256), (1, 40, 33, 7, 64, 0),
                                             (2, 30, 4, 2, 128, 112)])
def test_gradients_of_rows_without_a_token(sdl, t, gt, norm, weighted, B, T, Hq, Hk, d, rot):  # noqa: F811
    """Zeros, whatever the buffers held: an input that is not used has no gradient. Other rows on every call."""
    r = np.random.default_rng(41)
    q, qv = values(Hq, B, T, d, t, r, True)
    k, kv = values(Hk, B, T, d, t, r, False)
    gq, gqv = values(Hq, B, T, d, gt, r, False)
    gk, gkv = values(Hk, B, T, d, gt, r, True)
    kw, wq, wk = weights(norm, weighted, Hk, d, r)
    freq = BASE ** (-2 * np.arange(rot // 2) / max(rot, 1))
    f = make(sdl, True, norm, weighted, t, B, T, Hq, Hk, d, rot, token_major=T % 2 == 0, grad_dtype=DT[gt])
    for g in f.grads.values():
        if g is not None:
            g.fill_(7)
    for part in range(3):                                        # the third call has no tokens at all
        pos = np.arange(B * T).reshape(B, T) + 100
        pos[(np.arange(B * T) % 2 == part).reshape(B, T) | (part == 2)] = -1 - part
        p = torch.tensor(pos, dtype=torch.int32, device="cuda")
        got = f(*((gq, gk, p) if norm is None else (gq, gk, q, k, p)), **kw)
        live = (pos >= 0)[:, None, :, None]
        for n, g, x, w in (("q", gqv, qv, wq), ("k", gkv, kv, wk)):
            if g is None:
                continue
            dx, dw, edx, edw = ref.heads_grads(g, x, pos, freq, norm, 1e-6, w)
            near(got[n], np.where(live, dx, 0.0), edx * live, t, n)
            assert not got[n][torch.tensor(pos < 0, device="cuda")[:, None].expand(B, got[n].shape[1], T)].any()
            if dw is not None:
                near(got[n + "_weight"], dw, edw, "f32", n + "_weight")


# ---- features that are not rotated

@pytest.mark.parametrize("t", ["bf16", "f32"])
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("d,rot", [(64, 0), (64, 16), (64, 48), (128, 64), (256, 112), (32, 16)])
def test_not_finite_beside_the_rotated_part(sdl, t, interleaved, d, rot):  # noqa: F811
    """A feature behind the rotated part stays as it is and nobody else's, whatever its value, forwards and backwards."""
    B, T, H = 1, 5, 3
    r = np.random.default_rng(42)
    kw = dict(interleaved=interleaved, q_scale=0.25, rot_scale=1.1)
    f = make(sdl, False, None, False, t, B, T, H, 0, d, rot, **kw)
    b = make(sdl, True, None, False, t, B, T, H, 0, d, rot, **kw)
    x, _ = values(H, B, T, d, t, r, False)
    clean, back = f(x, None, first_position=9)[0].clone(), b(x, None, first_position=9)["q"].clone()
    assert torch.equal(clean[..., rot:], (0.25 * x[..., rot:].float()).to(x.dtype))      # one rounding of an exact product
    for i in {rot, rot + 1, (rot + d) // 2, d - 9, d - 1}:
        if i < rot:
            continue
        for value in (float("nan"), float("inf"), -float("inf")):
            z = x.clone()
            z[0, 1, 2, i] = value
            for got, want in ((f(z, None, first_position=9)[0], clean), (b(z, None, first_position=9)["q"], back)):
                want = want.clone()
                want[0, 1, 2, i] = value
                assert torch.equal(torch.nan_to_num(got, nan=12345.0), torch.nan_to_num(want, nan=12345.0)), (i, value)


# ---- angles

@pytest.mark.parametrize("interleaved", [False, True])
def test_angles_alone(sdl, interleaved):  # noqa: F811
    """Pairs (1, 0) come out as the cosine and the sine themselves: off by 2^-28 turns from the angle's conversion, 2^-33 from its
    last bit and a position times 2^-65 from the frequency's, and by a unit in the last place of sine and cosine."""
    from fractions import Fraction
    pi = Fraction(314159265358979323846264338327950288419716939937510582097494, 10 ** 59)
    T, d = 2000, 64
    r = np.random.default_rng(43)
    pos = np.concatenate([np.arange(500), r.integers(0, 2 ** 31, T - 502), [2 ** 31 - 1, 2 ** 30]])
    freq = sdl.rotary_frequencies(d, BASE).numpy()
    per = [Fraction(float(v)) / (2 * pi) for v in freq]
    turn = np.array([[float(v * int(p) % 1) for v in per] for p in pos])
    x = torch.zeros(1, 1, T, d, device="cuda")
    u, v = (slice(0, d, 2), slice(1, d, 2)) if interleaved else (slice(0, d // 2), slice(d // 2, d))
    x[..., u] = 1
    f = sdl.Rotary(torch.float32, 1, T, 1, 0, d, freq, interleaved=interleaved)
    y = f(x, None, torch.tensor(pos[None], dtype=torch.int32, device="cuda"))[0][0, 0].double().cpu().numpy()
    angle = 2 * np.pi * (2.0 ** -28 + 2.0 ** -33 + pos[:, None] * 2.0 ** -65)
    for got, want in ((y[:, u], np.cos(2 * np.pi * turn)), (y[:, v], np.sin(2 * np.pi * turn))):
        off = np.abs(got - want) - 2.0 ** -23 * np.abs(want)
        assert (off <= angle).all(), (off / angle).max()
