"""The recurrence of linear attention with one decay per head and its gradients, token by token in float64 (numpy).

    S_t = exp(g_t) S_{t-1} + k_t v_t^T,   o_t = S_t^T q_t

q, k [B,Hq,T,dk] (value head h reads head h // (H / Hq)), v [B,H,T,dv], g [B,H,T]. The gradients are the recurrence's own
reverse mode: dS_t = q_t dO_t^T + exp(g_{t+1}) dS_{t+1}, dq_t = S_t dO_t, dk_t = dS_t v_t, dv_t = dS_t^T k_t,
dg_t = exp(g_t) <S_{t-1}, dS_t>.
"""

import numpy as np


def _heads(x, H):
    return np.repeat(np.asarray(x, np.float64), H // x.shape[1], axis=1)


def forward(q, k, v, g, S0=None):
    """o [B,H,T,dv], S_T, and `size` [B,H,T,dv], the same with absolute values throughout (what roundings scale with)."""
    v, g = np.asarray(v, np.float64), np.asarray(g, np.float64)
    B, H, T, dv = v.shape
    q, k = _heads(q, H), _heads(k, H)
    dk = q.shape[-1]
    S = np.zeros((B, H, dk, dv)) if S0 is None else np.array(S0, np.float64)
    A = np.abs(S)
    o, size = np.zeros((B, H, T, dv)), np.zeros((B, H, T, dv))
    for t in range(T):
        e = np.exp(g[:, :, t])[..., None, None]
        S = e * S + k[:, :, t, :, None] * v[:, :, t, None, :]
        A = e * A + np.abs(k[:, :, t, :, None] * v[:, :, t, None, :])
        o[:, :, t] = np.einsum("bhi,bhij->bhj", q[:, :, t], S)
        size[:, :, t] = np.einsum("bhi,bhij->bhj", np.abs(q[:, :, t]), A)
    return o, S, size, A


def backward(q, k, v, g, dO, dST=None, S0=None):
    v, g, dO = (np.asarray(x, np.float64) for x in (v, g, dO))
    B, H, T, dv = v.shape
    Hq = q.shape[1]
    q, k = _heads(q, H), _heads(k, H)
    dk = q.shape[-1]
    S = np.zeros((T + 1, B, H, dk, dv))
    if S0 is not None:
        S[0] = S0
    for t in range(T):
        S[t + 1] = np.exp(g[:, :, t])[..., None, None] * S[t] + k[:, :, t, :, None] * v[:, :, t, None, :]
    R = np.zeros((B, H, dk, dv)) if dST is None else np.array(dST, np.float64)
    dq, dkey, dval, dg = np.zeros_like(q), np.zeros_like(k), np.zeros_like(v), np.zeros((B, H, T))
    for t in range(T - 1, -1, -1):
        R = R + q[:, :, t, :, None] * dO[:, :, t, None, :]
        dq[:, :, t] = np.einsum("bhij,bhj->bhi", S[t + 1], dO[:, :, t])
        dkey[:, :, t] = np.einsum("bhij,bhj->bhi", R, v[:, :, t])
        dval[:, :, t] = np.einsum("bhij,bhi->bhj", R, k[:, :, t])
        e = np.exp(g[:, :, t])
        dg[:, :, t] = e * np.einsum("bhij,bhij->bh", S[t], R)
        R = e[..., None, None] * R
    over = lambda x: x.reshape(B, Hq, H // Hq, T, -1).sum(2)  # noqa: E731
    return {"q": over(dq), "k": over(dkey), "v": dval, "decay": dg, "S0": R}


def plan(lengths, slots, context, capacity, block):
    """Tables of a ragged batch (valid lengths only)."""
    R = len(lengths)
    starts, block_starts = np.zeros(R + 1, np.int32), np.zeros(R + 1, np.int32)
    blocks = np.full((capacity // block + R, 4), -1, np.int32)
    token_slot, token_pos = np.full(capacity, -1, np.int32), np.full(capacity, -1, np.int32)
    nb = 0
    for r, n in enumerate(lengths):
        starts[r + 1] = starts[r] + n
        for i in range(0, n, block):
            blocks[nb] = (r, starts[r] + i, min(block, n - i), i // block)
            nb += 1
        block_starts[r + 1] = nb
        token_slot[starts[r]:starts[r + 1]] = slots[r]
        token_pos[starts[r]:starts[r + 1]] = context[r] + np.arange(n)
    return {"starts": starts, "blocks": blocks, "block_starts": block_starts, "token_slot": token_slot,
            "token_pos": token_pos}
