"""Linear attention with one decay per head: refusals of the C ABI (nothing is launched, no GPU), and the float64 reference
of the GPU tests against the framework's own oracle and against differences."""

import numpy as np
import pytest

import head_decay_reference as ref
import oracle

FAKE = 1 << 20   # aligned, never dereferenced: every check comes before the first launch


@pytest.fixture(scope="module")
def sdl():
    from structured_decay_linear_gb300 import build as nvbuild
    nvbuild.build()
    import structured_decay_linear_gb300 as s
    s.library()
    return s


def tensor(sdl, B, H, T, d, data=FAKE, **kw):
    v = dict(sb=H * T * d, sh=T * d, st=d)
    v.update(kw)
    return sdl.dplr_hd_tensor(data, v["sb"], v["sh"], v["st"])


@pytest.mark.parametrize("kw,expect", [
    (dict(), 0), (dict(q_heads=2), 0), (dict(q_heads=3), 1), (dict(q_heads=0), 1), (dict(T=0), 0), (dict(T=-1), 1),
    (dict(B=0), 1), (dict(dk=48), 2), (dict(dv=256), 2), (dict(dk=0), 1), (dict(B=1 << 14, H=1 << 10, T=1), 2),
    (dict(B=1, H=4, T=1 << 29), 2), (dict(dt="f32", dk=32, dv=32), 0)])
def test_descriptors(sdl, kw, expect):
    v = dict(B=2, H=4, T=100, dk=64, dv=128, dt="bf16", q_heads=None)
    v.update(kw)
    d = sdl.make_hd_desc(v["dt"], v["B"], v["H"], v["T"], v["dk"], v["dv"], v["q_heads"])
    assert sdl.dplr_hd_check(d) == expect
    sizes = (sdl.dplr_hd_workspace_size(d), sdl.dplr_hd_backward_workspace_size(d))
    assert all(n >= 256 and n % 256 == 0 for n in sizes) if expect == 0 else sizes == (0, 0)
    assert (sdl.dplr_hd_path(d) != "") == (expect == 0)


def test_bad_enums(sdl):
    d = sdl.make_hd_desc("bf16", 1, 1, 8, 64, 64)
    d.in_dtype = 7
    assert sdl.dplr_hd_check(d) == 1
    d = sdl.make_hd_desc("bf16", 1, 1, 8, 64, 64)
    d.per_head = 2
    assert sdl.dplr_hd_check(d) == 1
    assert sdl.library().dplr_hd_check(None) == 1


def forward(sdl, d, **kw):
    B, H, Hq, T, dk, dv = d.B, d.H, d.Hq, d.T, d.dk, d.dv
    a = dict(q=tensor(sdl, B, Hq, T, dk), k=tensor(sdl, B, Hq, T, dk), v=tensor(sdl, B, H, T, dv),
             decay=sdl.dplr_hd_tensor(FAKE, H * T, T, 1), S0=FAKE, o=tensor(sdl, B, H, T, dv), S_T=FAKE, ws=FAKE,
             nbytes=sdl.dplr_hd_workspace_size(d))
    a.update(kw)
    return sdl.dplr_hd_forward(d, a["q"], a["k"], a["v"], a["decay"], a["S0"], a["o"], a["S_T"], a["ws"], a["nbytes"],
                               None)


def test_forward_refuses(sdl):
    d = sdl.make_hd_desc("bf16", 2, 4, 100, 64, 128, 2)
    bad = lambda heads, dim: [  # noqa: E731
        None, tensor(sdl, 2, heads, 100, dim, data=None), tensor(sdl, 2, heads, 100, dim, data=FAKE + 8),
        tensor(sdl, 2, heads, 100, dim, sb=0), tensor(sdl, 2, heads, 100, dim, sh=-64),
        tensor(sdl, 2, heads, 100, dim, st=dim + 4)]
    for name, heads, dim in (("q", 2, 64), ("k", 2, 64), ("v", 4, 128), ("o", 4, 128)):
        for t in bad(heads, dim):
            assert forward(sdl, d, **{name: t}) == 1, name
        assert forward(sdl, d, **{name: tensor(sdl, 2, heads, 100, dim, sb=1 << 42)}) == 2
    assert forward(sdl, d, o=tensor(sdl, 2, 4, 100, 128, st=64)) == 1            # rows of o on top of each other
    assert forward(sdl, d, o=tensor(sdl, 2, 4, 100, 128, sh=99 * 128)) == 1
    for t in (None, sdl.dplr_hd_tensor(FAKE + 2, 400, 100, 1), sdl.dplr_hd_tensor(FAKE, 400, 100, -1),
              sdl.dplr_hd_tensor(FAKE, -400, 100, 1)):
        assert forward(sdl, d, decay=t) == 1
    assert forward(sdl, d, S0=FAKE + 4) == 1 and forward(sdl, d, S_T=FAKE + 8) == 1
    need = sdl.dplr_hd_workspace_size(d)
    assert forward(sdl, d, nbytes=need - 1) == 3 and forward(sdl, d, ws=None) == 3 and forward(sdl, d, ws=FAKE + 16) == 3


def test_backward_refuses(sdl):
    d = sdl.make_hd_desc("bf16", 2, 4, 100, 64, 128, 2)
    kq, vv = tensor(sdl, 2, 2, 100, 64), tensor(sdl, 2, 4, 100, 128)
    names = ["q", "k", "v", "decay", "S0", "dO", "dST", "dq", "dk", "dv", "ddecay", "dS0", "ws", "nbytes"]
    base = [kq, kq, vv, sdl.dplr_hd_tensor(FAKE, 400, 100, 1), FAKE, vv, FAKE, kq, kq, vv, FAKE, FAKE, FAKE,
            sdl.dplr_hd_backward_workspace_size(d)]

    def call(**kw):
        return sdl.dplr_hd_backward(d, *[kw.get(n, b) for n, b in zip(names, base)], None)

    for n in ("q", "k", "v", "decay", "dO", "dq", "dk", "dv"):
        assert call(**{n: None}) == 1, n
    for n in ("dq", "dk"):
        assert call(**{n: tensor(sdl, 2, 2, 100, 64, sh=64)}) == 1               # overlapping rows
    for n in ("S0", "dST", "dS0"):
        assert call(**{n: FAKE + 4}) == 1
    assert call(ddecay=FAKE + 2) == 1
    assert call(nbytes=base[-1] - 1) == 3 and call(ws=None) == 3 and call(ws=FAKE + 32) == 3


def test_plan_refuses(sdl):
    def call(R=4, cap=100, block=128, slots=8, **kw):
        names = ["lengths", "slots", "context", "starts", "blocks", "block_starts", "token_slot", "token_pos", "status"]
        return sdl.dplr_hd_plan(R, cap, block, slots, *[kw.get("p_" + n, FAKE) for n in names], None)

    assert call(R=0) == 1 and call(cap=-1) == 1 and call(block=0) == 1 and call(slots=0) == 1
    assert call(R=8193) == 2 and call(cap=1 << 30) == 2 and call(block=100) == 2 and call(slots=(1 << 20) + 1) == 2
    for n in ("lengths", "slots", "context", "starts", "blocks", "block_starts", "token_slot", "token_pos", "status"):
        assert call(**{"p_" + n: None}) == 1 and call(**{"p_" + n: FAKE + 2}) == 1, n
    assert call(p_blocks=FAKE + 4) == 1


def test_packed_and_decode_refuse(sdl):
    d = sdl.make_hd_desc("bf16", 1, 4, 100, 64, 128, 2)
    kq, vv, g = tensor(sdl, 1, 2, 100, 64), tensor(sdl, 1, 4, 100, 128), sdl.dplr_hd_tensor(FAKE, 0, 100, 1)
    assert sdl.dplr_hd_packed_workspace_size(d, 3, 100) == 0 and sdl.dplr_hd_packed_workspace_size(d, 0, 128) == 0
    assert sdl.dplr_hd_packed_workspace_size(sdl.make_hd_desc("bf16", 2, 4, 100, 64, 128, 2), 3, 128) == 0
    small, large = (sdl.dplr_hd_packed_workspace_size(d, 3, b) for b in (128, 64))
    assert small == 256 and large > (1 + 3) * 4 * 64 * 128 * 4

    def packed(R=3, block=64, slots=8, tables=(FAKE,) * 4, q=kq, k=kq, v=vv, decay=g, S=FAKE, o=vv, ws=FAKE, n=large):
        return sdl.dplr_hd_forward_packed(d, R, block, slots, *tables, q, k, v, decay, S, o, ws, n, None)

    for i in range(4):
        assert packed(tables=[None if j == i else FAKE for j in range(4)]) == 1
    assert packed(R=0) == 1 and packed(block=48) == 1 and packed(slots=0) == 1 and packed(S=None) == 1
    assert packed(q=None) == 1 and packed(o=None) == 1 and packed(decay=None) == 1 and packed(n=large - 1) == 3
    assert packed(S=FAKE + 4) == 1 and packed(ws=None) == 3

    one = sdl.make_hd_desc("bf16", 5, 4, 1, 64, 128, 2)
    kq, vv, g = tensor(sdl, 5, 2, 1, 64), tensor(sdl, 5, 4, 1, 128), sdl.dplr_hd_tensor(FAKE, 4, 1, 0)

    def decode(desc=one, n=8, slots=FAKE, q=kq, k=kq, v=vv, decay=g, S=FAKE, o=vv, status=None):
        return sdl.dplr_hd_decode_step(desc, n, slots, q, k, v, decay, S, o, status, None)

    assert decode(desc=d) == 1 and decode(n=0) == 1 and decode(slots=None) == 1 and decode(S=None) == 1
    assert decode(slots=FAKE + 1) == 1 and decode(status=FAKE + 1) == 1
    assert all(decode(**{n: None}) == 1 for n in ("q", "k", "v", "decay", "o"))


# ---- the reference itself

def inputs(B=1, H=2, Hq=2, T=20, dk=32, dv=32, seed=0):
    r = np.random.default_rng(seed)
    return dict(q=r.standard_normal((B, Hq, T, dk)), k=r.standard_normal((B, Hq, T, dk)) / dk ** 0.5,
                v=r.standard_normal((B, H, T, dv)), g=-0.3 * r.random((B, H, T)), S0=r.standard_normal((B, H, dk, dv)))


def test_reference_is_the_oracle_without_a_low_rank_term():
    """Generic mode with A = B = 0 and the same decay in every channel, float32 inputs (so that both read the same)."""
    x = {n: v.astype(np.float32) for n, v in inputs().items()}
    o, S, _, _ = ref.forward(**x)
    B, H, T, dk = x["q"].shape
    decay = np.broadcast_to(x["g"][..., None], (B, H, T, dk)).copy()
    zero = np.zeros((B, H, T, 1, dk), np.float32)
    o2, S2 = oracle.forward("generic", x["q"], None, None, decay, None, A=zero, Bm=zero, K=x["k"][:, :, :, None].copy(),
                            V=x["v"][:, :, :, None].copy(), S0=x["S0"])
    assert np.abs(o - o2).max() <= 1e-10 * np.abs(o).max() and np.abs(S - S2).max() <= 1e-10 * np.abs(S).max()


def test_reference_gradients_against_differences():
    x = inputs(H=4, Hq=2, T=7, dk=3, dv=5, seed=1)
    r = np.random.default_rng(2)
    dO, dST = r.standard_normal((1, 4, 7, 5)), r.standard_normal((1, 4, 3, 5))
    got = ref.backward(x["q"], x["k"], x["v"], x["g"], dO, dST, x["S0"])
    loss = lambda y: (ref.forward(**y)[0] * dO).sum() + (ref.forward(**y)[1] * dST).sum()  # noqa: E731
    for n, name in (("q", "q"), ("k", "k"), ("v", "v"), ("g", "decay"), ("S0", "S0")):
        u = r.standard_normal(x[n].shape)
        hi, lo = dict(x), dict(x)
        hi[n], lo[n] = x[n] + 1e-6 * u, x[n] - 1e-6 * u
        assert abs((loss(hi) - loss(lo)) / 2e-6 - (got[name] * u).sum()) <= 1e-6 * np.linalg.norm(got[name])


def test_default_block_of_a_ragged_batch(sdl):
    """A multiple of 32 that follows the tokens and heads that an SM gets: on the tensor cores the next power of two, at
    least 512; on the CUDA cores the last one, at least 128."""
    block = lambda dt, T, H: sdl.default_block(sdl.make_hd_desc(dt, 1, H, T, 128, 128))  # noqa: E731
    assert [block("bf16", T, 16) for T in (0, 1, 3000, 16203, 55165)] == [512, 512, 512, 2048, 8192]
    assert [block("f32", T, 16) for T in (0, 1, 3000, 10000, 55165)] == [128, 128, 256, 1024, 4096]


def test_outputs_on_top_of_inputs_are_refused(sdl):
    """A result fed back into the object that holds it; S_T alone may be S0 (run on the GPU)."""
    at = lambda i: FAKE + (i << 30)  # noqa: E731
    d = sdl.make_hd_desc("bf16", 2, 4, 100, 128, 128)
    t = [tensor(sdl, 2, 4, 100, 128, data=at(i)) for i in range(8)]
    g = sdl.dplr_hd_tensor(at(9), 400, 100, 1)
    for i in range(3):
        assert forward(sdl, d, q=t[0], k=t[1], v=t[2], o=t[i], decay=g, S0=at(10), S_T=at(11), ws=at(12)) == 1
    names = ["q", "k", "v", "decay", "S0", "dO", "dST", "dq", "dk", "dv", "ddecay", "dS0", "ws", "nbytes"]
    base = [t[0], t[1], t[2], g, at(10), t[3], at(11), t[4], t[5], t[6], at(13), at(14), at(12),
            sdl.dplr_hd_backward_workspace_size(d)]

    def backward(**kw):
        return sdl.dplr_hd_backward(d, *[kw.get(n, b) for n, b in zip(names, base)], None)

    for n in ("dq", "dk", "dv"):
        assert all(backward(**{n: t[i]}) == 1 for i in range(4)), n
    assert backward(dk=t[4]) == 1 and backward(dv=t[5]) == 1 and backward(dv=t[4]) == 1
    assert backward(dS0=at(10)) == 1 and backward(dS0=at(11)) == 1 and backward(ddecay=at(9)) == 1
    d = sdl.make_hd_desc("bf16", 1, 4, 100, 128, 128)
    t = [tensor(sdl, 1, 4, 100, 128, data=at(i)) for i in range(3)]
    n = sdl.dplr_hd_packed_workspace_size(d, 3, 64)
    one = sdl.make_hd_desc("bf16", 5, 4, 1, 128, 128)
    u = [tensor(sdl, 5, 4, 1, 128, data=at(i)) for i in range(3)]
    for i in range(3):
        assert sdl.dplr_hd_forward_packed(d, 3, 64, 8, *[at(4)] * 4, *t, g, at(5), t[i], at(6), n, None) == 1
        assert sdl.dplr_hd_decode_step(one, 8, at(4), *u, sdl.dplr_hd_tensor(at(9), 4, 1, 0), at(5), u[i], None, None) == 1


def test_sizes_beyond_32_bits_are_refused(sdl):
    """The C interface takes 32-bit sizes; one above would lose its upper bits on the way: a block of 2^32 + 128 would become
    one of 128, for which the tables made for it have no room."""
    torch = pytest.importorskip("torch")
    device = torch.device("cuda", 0)
    for kw in (dict(block=2 ** 32 + 128), dict(block=2 ** 31), dict(capacity=2 ** 32 + 5), dict(requests=2 ** 32 + 1),
               dict(slots=2 ** 32 + 3)):
        a = dict(requests=3, capacity=100, slots=4, block=128)
        a.update(kw)
        with pytest.raises(ValueError, match="32 bits"):
            sdl.RequestPlan(**a, device=device)
    for kw in (dict(T=2 ** 32 + 5), dict(B=2 ** 32 + 1), dict(q_heads=2 ** 33 + 4), dict(dk=2 ** 32 + 64)):
        a = dict(B=1, H=4, T=10, dk=64, dv=64, q_heads=None)
        a.update(kw)
        with pytest.raises(ValueError, match="32 bits"):
            sdl.make_hd_desc("bf16", a["B"], a["H"], a["T"], a["dk"], a["dv"], a["q_heads"])
    with pytest.raises(ValueError, match="32 bits"):
        sdl.HeadDecayDecode(torch.bfloat16, 3, 4, 64, 64, 2 ** 32 + 3, device=device)


def test_workspace_of_a_ragged_batch_is_counted_without_overflow(sdl):
    """R requests and T / block blocks more may pass 31 bits: states and gate sums of all of them, 256-byte aligned."""
    d = sdl.make_hd_desc("f32", 1, 2, 1 << 20, 64, 32)
    for R in (1, 8192, 2 ** 31 - 32768, 2 ** 31 - 1):
        n = ((1 << 20) // 32 + R) * 2
        up = lambda x: -(-x // 256) * 256  # noqa: E731
        assert sdl.dplr_hd_packed_workspace_size(d, R, 32) == up(up(256 + n * 64 * 32 * 4) + n * 4)


def test_every_output_on_top_of_another_tensor_is_refused(sdl):
    """All pairs of an output and another tensor that start at the same address, for each call. (S_T may be S0.)"""
    at = lambda i: FAKE + (i << 30)  # noqa: E731
    d = sdl.make_hd_desc("bf16", 2, 4, 100, 128, 128)
    one = sdl.make_hd_desc("bf16", 5, 4, 1, 128, 128)
    ragged = sdl.make_hd_desc("bf16", 1, 4, 100, 128, 128)

    def row(desc, p):
        return tensor(sdl, desc.B, 4, desc.T, 128, data=p)

    def gates(desc, p):
        return sdl.dplr_hd_tensor(p, 4 * desc.T, desc.T, 1)

    def forward_call(q, k, v, decay, S0, o, S_T, ws):
        r = lambda p: row(d, p)  # noqa: E731
        return sdl.dplr_hd_forward(d, r(q), r(k), r(v), gates(d, decay), S0, r(o), S_T, ws, sdl.dplr_hd_workspace_size(d),
                                   None)

    def backward_call(q, k, v, decay, S0, dO, dST, dq, dk, dv, ddecay, dS0, ws):
        r = lambda p: row(d, p)  # noqa: E731
        return sdl.dplr_hd_backward(d, r(q), r(k), r(v), gates(d, decay), S0, r(dO), dST, r(dq), r(dk), r(dv), ddecay, dS0,
                                    ws, sdl.dplr_hd_backward_workspace_size(d), None)

    def packed_call(blocks, block_starts, slots, context, q, k, v, decay, S, o, ws):
        r = lambda p: row(ragged, p)  # noqa: E731
        return sdl.dplr_hd_forward_packed(ragged, 3, 64, 8, blocks, block_starts, slots, context, r(q), r(k), r(v),
                                          gates(ragged, decay), S, r(o), ws,
                                          sdl.dplr_hd_packed_workspace_size(ragged, 3, 64), None)

    def decode_call(slots, q, k, v, decay, S, o, status):
        r = lambda p: row(one, p)  # noqa: E731
        return sdl.dplr_hd_decode_step(one, 8, slots, r(q), r(k), r(v), gates(one, decay), S, r(o), status, None)

    def plan_call(lengths, slots, context, starts, blocks, block_starts, token_slot, token_pos, status):
        return sdl.dplr_hd_plan(4, 100, 128, 8, lengths, slots, context, starts, blocks, block_starts, token_slot, token_pos,
                                status, None)

    for call, outputs in ((forward_call, "o S_T"), (backward_call, "dq dk dv ddecay dS0"), (packed_call, "S o"),
                          (decode_call, "S o status"),
                          (plan_call, "starts blocks block_starts token_slot token_pos status")):
        names = call.__code__.co_varnames[:call.__code__.co_argcount]
        for out in outputs.split():
            for other in names:
                if other != out and {out, other} != {"S_T", "S0"}:
                    p = {n: at(i) for i, n in enumerate(names)}
                    p[out] = p[other]
                    assert call(**p) == 1, (call.__name__, out, other)
