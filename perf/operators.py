"""Cases that measure the linear attention with one decay per head and what serves it.

The operator, per batch b and value head h (state S in R^{dk x dv}, log-gate g_t <= 0):

    S_t = exp(g_t) S_{t-1} + k_t v_t^T,      o_t = S_t^T q_t

Five calls are measured: the prompt forward on equal lengths ("forward"), its gradients ("backward"), the tables of a
ragged batch built on the GPU ("plan"), the prompt forward of such a batch on a pool of states ("packed"), and the
one-token step on that pool ("decode"). Where `own` is false, `run` computes them with elementary torch operations in
32 bits (64 for sums of gates); where it is true it calls this package.
"""

import torch

own = False

F32, F64, I32 = torch.float32, torch.float64, torch.int32
TYPES = {"bf16": torch.bfloat16, "f32": torch.float32}


def listed():
    c = []
    # a short prompt of one user: launch latency counts
    c.append(dict(name="forward short", op="forward", dtype="bf16", B=1, H=16, Hq=16, T=100, dk=128, dv=128,
                  per_head=False, state=False, token_major=True))
    # the repository's benchmark sizes, gates learned per token, tensors as the projections leave them
    c.append(dict(name="forward B8 T8192", op="forward", dtype="bf16", B=8, H=16, Hq=16, T=8192, dk=128, dv=128,
                  per_head=False, state=False, token_major=True))
    # one long document continued from a state, a fixed decay per head: few heads, so the sequence itself is split
    c.append(dict(name="forward B1 T32768", op="forward", dtype="bf16", B=1, H=16, Hq=16, T=32768, dk=128, dv=128,
                  per_head=True, state=True, token_major=False))
    # 32-bit inputs at the generic configuration's head sizes, odd length
    c.append(dict(name="forward f32 T2001", op="forward", dtype="f32", B=2, H=8, Hq=8, T=2001, dk=64, dv=64,
                  per_head=False, state=True, token_major=False))
    # prompts of 32 requests of different lengths in one call, four query/key heads shared by 16 value heads
    c.append(dict(name="packed 32 requests", op="packed", dtype="bf16", R=32, longest=2000, spare=100, H=16, Hq=4,
                  dk=128, dv=64, slots=48, per_head=False))
    # a batch of short requests
    c.append(dict(name="packed 100 short", op="packed", dtype="bf16", R=100, longest=60, spare=0, H=16, Hq=16,
                  dk=128, dv=128, slots=128, per_head=True))
    # a training step's gradients
    c.append(dict(name="backward B4 T4096", op="backward", dtype="bf16", B=4, H=16, Hq=16, T=4096, dk=128, dv=128,
                  per_head=False, state=False, token_major=True))
    # 32-bit gradients, odd length, shared query/key heads, a state carried in and out
    c.append(dict(name="backward f32 T777", op="backward", dtype="f32", B=2, H=8, Hq=2, T=777, dk=64, dv=64,
                  per_head=False, state=True, token_major=False))
    # tokens of a few users, and of a large serving batch with rows that hold no request
    c.append(dict(name="decode 8 rows", op="decode", dtype="bf16", N=8, H=16, Hq=16, dk=128, dv=128, slots=8, idle=0,
                  per_head=False))
    c.append(dict(name="decode 256 rows", op="decode", dtype="bf16", N=256, H=16, Hq=16, dk=128, dv=128, slots=300,
                  idle=7, per_head=False))
    # tables of a scheduler's step: a few requests, and 1500 with about 200 thousand tokens
    c.append(dict(name="plan 12 requests", op="plan", R=12, longest=200, spare=50, slots=16, block=128))
    c.append(dict(name="plan 1500 requests", op="plan", R=1500, longest=270, spare=5000, slots=2048, block=128))
    return c


def draw(rng):
    def size(lo, hi):
        return int(round(lo * (hi / lo) ** rng.random()))

    op = rng.choice(["forward", "forward", "packed", "backward", "decode", "plan"])
    H = rng.choice([1, 2, 3, 4, 6, 8, 16])
    Hq = rng.choice([h for h in (1, 2, 3, 4, 6, 8, 16) if H % h == 0])
    dtype = rng.choice(["bf16", "bf16", "f32"])
    dk, dv = rng.choice([32, 64, 128, 128]), rng.choice([32, 64, 128, 128])
    per_head = rng.random() < 0.4
    base = dict(op=op, dtype=dtype, H=H, Hq=Hq, dk=dk, dv=dv, per_head=per_head)
    if op in ("forward", "backward"):
        most = 16384 if op == "forward" and dtype == "bf16" else 4096
        T = size(1, most)
        B = rng.randint(1, max(1, min(8, (200000 if dtype == "bf16" else 40000) // (H * T))))
        return dict(base, B=B, T=T, state=rng.random() < 0.5, token_major=rng.random() < 0.5)
    if op == "packed":
        R, longest = size(1, 100), size(1, 2000)
        while R * longest > 40000:
            longest = max(1, longest // 2)
        return dict(base, R=R, longest=longest, spare=rng.choice([0, 0, 33, 200]), slots=R + rng.randint(0, 20))
    if op == "decode":
        N = size(1, 256)
        return dict(base, N=N, slots=N + rng.randint(0, 40), idle=rng.randint(0, N // 8))
    R = size(1, 2000)
    return dict(op="plan", R=R, longest=size(1, 270), spare=rng.randint(0, 3000), slots=R + rng.randint(0, 300),
                block=rng.choice([64, 128, 256, 1024]))


# ---------------------------------------------------------------------------------------------------------------
# inputs
# ---------------------------------------------------------------------------------------------------------------

def capacity_of(case):
    """Rows that the program reserves for a batch: a little over what such a batch has."""
    return case["R"] * case["longest"] // 2 + case["longest"] + case["spare"]


def lengths_of(case, seed):
    """Lengths of a ragged batch from the seed: 0 (a request without new tokens) to the longest, which one has; what
    goes beyond the capacity waits for another step."""
    g = torch.Generator().manual_seed(1000003 * seed + 17)
    n = torch.randint(1, case["longest"] + 1, (case["R"],), generator=g)
    n[torch.rand(case["R"], generator=g) < 0.05] = 0
    n[int(torch.randint(0, case["R"], (1,), generator=g))] = case["longest"]
    return torch.minimum(n, (capacity_of(case) - n.cumsum(0) + n).clamp(min=0))


def gates(case, shape_token, H, gen):
    """Log-gates: a fixed rate per head between 1/16 and 1/1024, or learned ones around such rates."""
    h = torch.arange(H, device="cuda", dtype=F32)
    rate = torch.exp2(-4 - 6 * h / max(H - 1, 1))
    if case["per_head"]:
        return -rate * (1 + 0.2 * torch.rand(H, device="cuda", generator=gen))
    x = torch.randn(shape_token, device="cuda", generator=gen)
    return -rate * torch.nn.functional.softplus(x) * 1.5     # the last axis but one or the axis of heads is last


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    rn = lambda *s: torch.randn(*s, device="cuda", generator=gen)  # noqa: E731
    st = {"case": case}
    if case["op"] in ("plan", "packed"):
        n = lengths_of(case, seed)
        g = torch.Generator().manual_seed(seed + 5)
        st["lengths"] = n.to("cuda", I32)
        st["slot"] = torch.randperm(case["slots"], generator=g)[:case["R"]].to("cuda", I32)
        context = torch.randint(0, 3, (case["R"],), generator=g) * torch.randint(0, 5000, (case["R"],), generator=g)
        st["context"] = context.to("cuda", I32)
        st["capacity"] = capacity_of(case)
        st["longest"] = case["longest"]
    if case["op"] == "plan":
        if own:
            import structured_decay_linear_gb300 as sdl
            st["plan"] = sdl.RequestPlan(case["R"], st["capacity"], case["slots"], block=case["block"])
        return st
    dt, H, Hq, dk, dv = TYPES[case["dtype"]], case["H"], case["Hq"], case["dk"], case["dv"]

    def tokens(*lead, heads, d, unit=False, scale=1.0, major=False):
        """[B,H,T,d] (or [N,H,d]) values; `major`: stored with the token axis before the heads."""
        x = rn(*lead, heads, d) if major or len(lead) == 1 else rn(lead[0], heads, lead[1], d)
        x = torch.nn.functional.normalize(x, dim=-1) if unit else x * scale
        x = x.to(dt)
        return x.transpose(1, 2) if major else x

    if case["op"] in ("forward", "backward"):
        B, T, major = case["B"], case["T"], case["token_major"]
        st["q"] = tokens(B, T, heads=Hq, d=dk, scale=dk ** -0.5, major=major)
        st["k"] = tokens(B, T, heads=Hq, d=dk, unit=True, major=major)
        st["v"] = tokens(B, T, heads=H, d=dv, major=major)
        x = gates(case, (B, T, H), H, gen)
        st["decay"] = x if case["per_head"] else (x.transpose(1, 2) if major else x.transpose(1, 2).contiguous())
        st["S0"] = 0.1 * rn(B, H, dk, dv) if case["state"] else None
        if case["op"] == "backward":
            st["dO"] = tokens(B, T, heads=H, d=dv, major=major)
            st["dST"] = 0.1 * rn(B, H, dk, dv) if case["state"] else None
        if own:
            import structured_decay_linear_gb300 as sdl
            make = sdl.HeadDecay if case["op"] == "forward" else sdl.HeadDecayBackward
            st["call"] = make(dt, B, H, T, dk, dv, q_heads=Hq, per_head=case["per_head"], token_major=major)
        return st
    n = st["capacity"] if case["op"] == "packed" else case["N"]
    st["q"] = tokens(n, heads=Hq, d=dk, scale=dk ** -0.5)
    st["k"] = tokens(n, heads=Hq, d=dk, unit=True)
    st["v"] = tokens(n, heads=H, d=dv)
    st["decay"] = gates(case, (n, H), H, gen)
    st["S"] = 0.1 * rn(case["slots"], H, dk, dv)
    if case["op"] == "decode":
        g = torch.Generator().manual_seed(seed + 6)
        slot = torch.randperm(case["slots"], generator=g)[:n]
        slot[torch.randperm(n, generator=g)[:case["idle"]]] = -1
        st["slot"] = slot.to("cuda", I32)
        if own:
            import structured_decay_linear_gb300 as sdl
            st["call"] = sdl.HeadDecayDecode(dt, n, H, dk, dv, case["slots"], q_heads=Hq, per_head=case["per_head"])
    elif own:
        import structured_decay_linear_gb300 as sdl
        st["call"] = sdl.HeadDecayPacked(dt, case["R"], n, case["slots"], H, dk, dv, q_heads=Hq,
                                         per_head=case["per_head"])
    return st


# ---------------------------------------------------------------------------------------------------------------
# plain forms
# ---------------------------------------------------------------------------------------------------------------

def chunk_of(T):
    return 64 if T <= 8192 else 256


def heads_of(x, H):
    """[B,Hq,T,d] -> [B,H,T,d] fp32: query/key head h // (H / Hq) serves value head h."""
    return x.float().repeat_interleave(H // x.shape[1], dim=1)


def plain_scan(x, y, z, g, S0):
    """o_t = (sum_{u<=t} e^{g_{u+1}+..+g_t} y_u z_u^T + e^{g_1+..+g_t} S0)^T x_t, chunkwise, every step a batched operation.

    x, y [B,H,T,dx], z [B,H,T,dz] fp32, g [B,H,T] fp64; T a multiple of the chunk. Returns o and the states at every
    chunk boundary [B,H,N+1,dx,dz]."""
    B, H, T, dx = x.shape
    C = min(chunk_of(T), T)
    N, dz = T // C, z.shape[3]
    cut = lambda t: t.reshape(B, H, N, C, -1)  # noqa: E731
    x, y, z = cut(x), cut(y), cut(z)
    G = g.reshape(B, H, N, C).cumsum(-1)
    causal = torch.ones(C, C, dtype=torch.bool, device=x.device).tril()
    D = (G.unsqueeze(-1) - G.unsqueeze(-2)).float().masked_fill(~causal, float("-inf")).exp()
    o = ((x @ y.transpose(-1, -2)) * D) @ z
    total = G[..., -1]
    local = (y * (total.unsqueeze(-1) - G).float().exp().unsqueeze(-1)).transpose(-1, -2) @ z
    across = torch.nn.functional.pad(total.cumsum(-1), (1, 0))                       # [B,H,N+1]
    later = torch.ones(N + 1, N, dtype=torch.bool, device=x.device).tril(-1)
    A = (across.unsqueeze(-1) - across[..., 1:].unsqueeze(-2)).float().masked_fill(~later, float("-inf")).exp()
    S = (A @ local.reshape(B, H, N, dx * dz)).reshape(B, H, N + 1, dx, dz)
    if S0 is not None:
        S = S + across.float().exp()[..., None, None] * S0.unsqueeze(2)
    o = o + G.float().exp().unsqueeze(-1) * (x @ S[:, :, :-1])
    return o.reshape(B, H, T, dz), S


def padded(T, *xs):
    """Each [B,H,T,...] with zeros behind, to a multiple of the chunk."""
    C = min(chunk_of(T), T)
    more = -T % C
    return [torch.nn.functional.pad(x, (0, 0) * (x.dim() - 3) + (0, more)) for x in xs]


def full_gates(st, shape):
    g = st["decay"].double()
    return g[None, :, None].expand(shape) if st["case"]["per_head"] else g


def plain_forward(st):
    c = st["case"]
    B, H, T = c["B"], c["H"], c["T"]
    q, k, v, g = padded(T, heads_of(st["q"], H), heads_of(st["k"], H), st["v"].float(), full_gates(st, (B, H, T)))
    o, S = plain_scan(q, k, v, g, st["S0"])
    return {"o": o[:, :, :T].to(st["q"].dtype), "S": S[:, :, -1]}


def plain_backward(st):
    """The gradients are the same operator on other operands: dq = op(dO, v, k) with the states transposed, and
    backwards in time dk = op(v, dO, q), dv = op(k, q, dO), where the gate of token t+1 stands before token t."""
    c = st["case"]
    B, H, T, Hq = c["B"], c["H"], c["T"], c["Hq"]
    dt = st["q"].dtype
    q, k, v, dO, g = padded(T, heads_of(st["q"], H), heads_of(st["k"], H), st["v"].float(), st["dO"].float(),
                            full_gates(st, (B, H, T)))
    flip = lambda x: x.flip(2)  # noqa: E731
    tr = lambda S: None if S is None else S.transpose(-1, -2)  # noqa: E731
    back = torch.nn.functional.pad(flip(g)[:, :, :-1], (1, 0))
    dq, S = plain_scan(dO, v, k, g, tr(st["S0"]))
    dk, R = plain_scan(flip(v), flip(dO), flip(q), back, tr(st["dST"]))
    dv, dS = plain_scan(flip(k), flip(q), flip(dO), back, st["dST"])
    dk, dv = flip(dk), flip(dv)
    N = S.shape[2] - 1
    C = q.shape[2] // N
    # the gradient of the log-gates: within a chunk the suffix sums of q.dq - k.dk, onto <S, dS> at the chunk's end
    next_gate = torch.nn.functional.pad(g, (0, 1))[:, :, C::C]                       # the gate behind each chunk
    ends = next_gate.exp() * (S[:, :, 1:].double() * R.flip(2)[:, :, 1:].double()).sum((-1, -2))
    a = ((q * dq).sum(-1, dtype=F64) - (k * dk).sum(-1, dtype=F64)).reshape(B, H, N, C)
    dg = (a.flip(-1).cumsum(-1).flip(-1) + ends.unsqueeze(-1)).reshape(B, H, N * C)[:, :, :T]
    dg = dg.sum((0, 2)) if c["per_head"] else dg
    over = lambda x: x[:, :, :T].reshape(B, Hq, H // Hq, T, -1).sum(2).to(dt)  # noqa: E731
    first = g[:, :, 0].float().exp()[..., None, None]
    return {"q": over(dq), "k": over(dk), "v": dv[:, :, :T].to(dt), "decay": dg.float(), "S0": first * dS[:, :, -1]}


def plain_tables(st):
    """Starts of the requests, their blocks of `block` tokens, and each token's slot and position."""
    c = st["case"]
    n, cap, R = st["lengths"].long(), st["capacity"], st["case"]["R"]
    ends = n.cumsum(0)
    starts = torch.nn.functional.pad(ends, (1, 0))
    block = c["block"]
    most = cap // block + R
    blocks_of = (n + block - 1) // block
    block_ends = blocks_of.cumsum(0)
    i = torch.arange(most, device="cuda")
    r = torch.searchsorted(block_ends, i, right=True)
    live = i < block_ends[-1]
    r = r.clamp(max=R - 1)
    at = i - (block_ends - blocks_of)[r]
    size = torch.minimum(n[r] - at * block, torch.full_like(at, block))
    rows = torch.stack([r, starts[r] + at * block, size, at], 1)
    rows = torch.where(live[:, None], rows, torch.full_like(rows, -1))
    t = torch.arange(cap, device="cuda")
    rt = torch.searchsorted(ends, t, right=True)
    live = t < ends[-1]
    rt = rt.clamp(max=R - 1)
    none = torch.full_like(t, -1)
    return {"starts": starts.to(I32), "blocks": rows.to(I32),
            "block_starts": torch.nn.functional.pad(block_ends, (1, 0)).to(I32),
            "token_slot": torch.where(live, st["slot"].long()[rt], none).to(I32),
            "token_pos": torch.where(live, st["context"].long()[rt] + t - starts[rt], none).to(I32)}


def plain_packed(st):
    c = st["case"]
    R, L, H = c["R"], st["longest"], c["H"]
    n = st["lengths"].long()
    starts = torch.nn.functional.pad(n.cumsum(0), (1, 0))[:-1]
    at = starts[:, None] + torch.arange(L, device="cuda")
    live = torch.arange(L, device="cuda") < n[:, None]
    at = torch.where(live, at, torch.zeros_like(at))
    rows = lambda x: (x[at] * live[..., None, None]).transpose(1, 2)  # noqa: E731  [R,H,L,d]
    g = (st["decay"].double().expand(st["capacity"], H) if c["per_head"] else st["decay"].double())[at]
    g = (g * live[..., None]).transpose(1, 2)
    slot = st["slot"].long()
    S0 = st["S"][slot] * (st["context"] > 0)[:, None, None, None]
    q, k, v, g = padded(L, heads_of(rows(st["q"]), H), heads_of(rows(st["k"]), H), rows(st["v"]).float(), g)
    o, S = plain_scan(q, k, v, g, S0)
    has = n > 0
    st["S"][slot] = torch.where(has[:, None, None, None], S[:, :, -1], st["S"][slot])
    out = torch.zeros(st["capacity"], H, c["dv"], device="cuda", dtype=st["q"].dtype)
    out[at[live]] = o[:, :, :L].transpose(1, 2)[live].to(out.dtype)
    return {"o": out, "S": st["S"]}


def plain_decode(st):
    c = st["case"]
    slot = st["slot"].long()
    live = slot >= 0
    at = slot.clamp(min=0)
    group = c["H"] // c["Hq"]
    q, k = (st[x].float().repeat_interleave(group, dim=1) for x in ("q", "k"))
    e = st["decay"].float().exp()
    e = (e[None].expand(c["N"], -1) if c["per_head"] else e)[..., None, None]
    S = e * st["S"][at] + k.unsqueeze(-1) * st["v"].float().unsqueeze(-2)
    o = (q.unsqueeze(-2) @ S).squeeze(-2) * live[:, None, None]
    keep = torch.where(live, at, torch.full_like(at, c["slots"]))
    pool = torch.cat([st["S"], st["S"][:1]])                        # idle rows go to a spare row behind the pool
    pool[keep] = S
    st["S"].copy_(pool[:-1])
    return {"o": o.to(st["q"].dtype), "S": st["S"]}


def run(st):
    op = st["case"]["op"]
    if not own:
        return {"forward": plain_forward, "backward": plain_backward, "plan": plain_tables, "packed": plain_packed,
                "decode": plain_decode}[op](st)
    if op == "forward":
        o, S_T = st["call"](st["q"], st["k"], st["v"], st["decay"], S0=st["S0"])
        return {"o": o, "S": S_T}
    if op == "backward":
        return st["call"](st["dO"], st["dST"], st["q"], st["k"], st["v"], st["decay"], S0=st["S0"])
    if op == "plan":
        return st["plan"](st["lengths"], st["slot"], st["context"])
    if op == "packed":
        call = st["call"]
        call.plan(st["lengths"], st["slot"], st["context"])
        return {"o": call(st["q"], st["k"], st["v"], st["decay"], st["S"]), "S": st["S"]}
    return {"o": st["call"](st["q"], st["k"], st["v"], st["decay"], st["S"], st["slot"]), "S": st["S"]}


# ---------------------------------------------------------------------------------------------------------------
# what a pass cannot do without
# ---------------------------------------------------------------------------------------------------------------

def work(case):
    if case["op"] == "plan":
        tokens = capacity_of(case)
        return {"bytes": 4.0 * (3 * case["R"] + 2 * (case["R"] + 1) + 4 * (tokens // case["block"] + case["R"]) +
                                2 * tokens), "flops": 0.0}
    es = 2 if case["dtype"] == "bf16" else 4
    H, Hq, dk, dv = case["H"], case["Hq"], case["dk"], case["dv"]
    state = 4.0 * H * dk * dv
    if case["op"] == "packed":
        rows, states = 0.5 * case["R"] * case["longest"], 1.7 * case["R"]
    elif case["op"] == "decode":
        rows, states = case["N"], 2.0 * (case["N"] - case["idle"])
    else:
        rows, states = case["B"] * case["T"], case["B"] * (2 if case["state"] else 1)
    gate = 4.0 * H * (0 if case["per_head"] else 1)
    if case["op"] == "backward":
        states = case["B"] * (3 if case["state"] else 1)
        return {"bytes": rows * (es * (4 * Hq * dk + 3 * H * dv) + 2 * gate) + states * state,
                "flops": 10.0 * rows * H * dk * dv}
    return {"bytes": rows * (es * (2 * Hq * dk + 2 * H * dv) + gate) + states * state, "flops": 4.0 * rows * H * dk * dv}


# ---------------------------------------------------------------------------------------------------------------
# the definition in 64 bits: the recurrence, token by token
# ---------------------------------------------------------------------------------------------------------------

def exact(case, seed):
    global own
    kept, own = own, False
    st = prepare(case, seed)
    own = kept
    op = case["op"]
    if op == "plan":
        return None
    H = case["H"]
    group = H // case["Hq"]
    if op == "decode":
        S, o = st["S"].double(), torch.zeros(case["N"], H, case["dv"], device="cuda", dtype=F64)
        q, k = (st[x].double().repeat_interleave(group, dim=1) for x in ("q", "k"))
        e = st["decay"].double().exp().expand(case["N"], H)
        for row, s in enumerate(st["slot"].tolist()):
            if s >= 0:
                S[s] = e[row][:, None, None] * S[s] + torch.einsum("hi,hj->hij", k[row], st["v"][row].double())
                o[row] = torch.einsum("hi,hij->hj", q[row], S[s])
        return {"o": o, "S": S}
    if op == "packed":
        S, o = st["S"].double(), torch.zeros(st["capacity"], H, case["dv"], device="cuda", dtype=F64)
        n, slot = st["lengths"].tolist(), st["slot"].long()
        first = torch.tensor([sum(n[:r]) for r in range(len(n))], device="cuda")
        cur = S[slot]
        cur[st["context"] == 0] = 0
        size = st["lengths"].long()
        decay = st["decay"].double().expand(st["capacity"], H)
        for t in range(max(n)):
            r = torch.nonzero(size > t).flatten()
            at = first[r] + t
            q, k = (st[x][at].double().repeat_interleave(group, dim=1) for x in ("q", "k"))
            new = decay[at].exp()[..., None, None] * cur[r] + k.unsqueeze(-1) * st["v"][at].double().unsqueeze(-2)
            cur[r] = new
            o[at] = (q.unsqueeze(-2) @ new).squeeze(-2)
        has = size > 0
        S[slot[has]] = cur[has]
        return {"o": o, "S": S}
    B, T, dk, dv = case["B"], case["T"], case["dk"], case["dv"]
    flat = lambda x: x.double().reshape(B * H, T, -1).transpose(0, 1).contiguous()  # noqa: E731  [T,BH,d]
    q, k = (flat(st[x].repeat_interleave(group, dim=1)) for x in ("q", "k"))
    v = flat(st["v"])
    decay = st["decay"].double()
    g = flat((decay[None, :, None].expand(B, H, T) if case["per_head"] else decay).unsqueeze(-1))   # [T,BH,1]
    e = g.exp().unsqueeze(-1)
    zero = torch.zeros(B, H, dk, dv, device="cuda", dtype=F64)
    S = (zero if st["S0"] is None else st["S0"].double()).reshape(B * H, dk, dv).clone()
    shaped = lambda x: x.transpose(0, 1).reshape(B, H, T, -1)  # noqa: E731
    if op == "forward":
        o = torch.empty(T, B * H, dv, device="cuda", dtype=F64)
        for t in range(T):
            S.mul_(e[t]).baddbmm_(k[t].unsqueeze(-1), v[t].unsqueeze(-2))
            torch.bmm(q[t].unsqueeze(-2), S, out=o[t].unsqueeze(-2))
        return {"o": shaped(o), "S": S.reshape(B, H, dk, dv)}
    dO = flat(st["dO"])
    R = (zero if st["dST"] is None else st["dST"].double()).reshape(B * H, dk, dv).clone()
    dq, dkey, dval = torch.empty_like(q), torch.empty_like(k), torch.empty_like(v)
    for t in range(T):
        S.mul_(e[t]).baddbmm_(k[t].unsqueeze(-1), v[t].unsqueeze(-2))
        torch.bmm(S, dO[t].unsqueeze(-1), out=dq[t].unsqueeze(-1))
    end = (S * R).sum((-1, -2))
    for t in range(T - 1, -1, -1):
        R.baddbmm_(q[t].unsqueeze(-1), dO[t].unsqueeze(-2))
        torch.bmm(R, v[t].unsqueeze(-1), out=dkey[t].unsqueeze(-1))
        torch.bmm(k[t].unsqueeze(-2), R, out=dval[t].unsqueeze(-2))
        R.mul_(e[t])
    a = (q * dq).sum(-1) - (k * dkey).sum(-1)                                         # [T,BH]
    dg = shaped((a.flip(0).cumsum(0).flip(0) + end).unsqueeze(-1)).squeeze(-1)
    over = lambda x: shaped(x).reshape(B, H // group, group, T, -1).sum(2)  # noqa: E731
    return {"q": over(dq), "k": over(dkey), "v": shaped(dval), "decay": dg.sum((0, 2)) if case["per_head"] else dg,
            "S0": R.reshape(B, H, dk, dv)}
