"""Linear attention with a decay per head, row by row in 64 bits.

    S_t = exp(log_decay_h) S_{t-1} + k_t v_t^T,   o_t = scale S_t^T q_t

per user and head, and its gradients by the transposed recurrence

    G_t = q_t (scale do_t)^T + exp(log_decay_h) G_{t+1},   G_{n+1} term = dS_n
    dq_t = scale S_t do_t,  dk_t = G_t v_t,  dv_t = G_t^T k_t,  dS_0 = exp(log_decay_h) G_1

where dS_n enters G_n undecayed.
"""

from __future__ import annotations

import numpy as np


def _states(heads, dk, dv, initial, user):
    return np.zeros((heads, dk, dv)) if initial is None else np.array(initial[user], np.float64)


def linear_attention(q, k, v, log_decay, offsets, scale, initial_state=None):
    """(out (N, H, dv), final_state (B, H, dk, dv)); rows of no user are zero."""
    q, k, v = (np.asarray(x, np.float64) for x in (q, k, v))
    decay = np.exp(np.asarray(log_decay, np.float64))[:, None, None]
    heads, dk, dv = q.shape[1], q.shape[2], v.shape[2]
    out, finals = np.zeros((q.shape[0], heads, dv)), []
    for b in range(len(offsets) - 1):
        S = _states(heads, dk, dv, initial_state, b)
        for t in range(offsets[b], offsets[b + 1]):
            S = decay * S + k[t][:, :, None] * v[t][:, None, :]
            out[t] = scale * np.einsum("hd,hde->he", q[t], S)
        finals.append(S)
    return out, np.array(finals).reshape(len(offsets) - 1, heads, dk, dv)


def linear_attention_grad(q, k, v, log_decay, offsets, scale, d_out, initial_state=None,
                          d_final_state=None):
    """dict(dq, dk, dv, d_initial_state)."""
    q, k, v, d_out = (np.asarray(x, np.float64) for x in (q, k, v, d_out))
    decay = np.exp(np.asarray(log_decay, np.float64))[:, None, None]
    heads, dk, dv = q.shape[1], q.shape[2], v.shape[2]
    g = dict(dq=np.zeros_like(q), dk=np.zeros_like(k), dv=np.zeros_like(v))
    starts = []
    for b in range(len(offsets) - 1):
        rows = range(offsets[b], offsets[b + 1])
        S = _states(heads, dk, dv, initial_state, b)
        for t in rows:
            S = decay * S + k[t][:, :, None] * v[t][:, None, :]
            g["dq"][t] = scale * np.einsum("hde,he->hd", S, d_out[t])
        G = _states(heads, dk, dv, d_final_state, b)
        for t in reversed(rows):
            G = G + scale * q[t][:, :, None] * d_out[t][:, None, :]
            g["dk"][t] = np.einsum("hde,he->hd", G, v[t])
            g["dv"][t] = np.einsum("hde,hd->he", G, k[t])
            G = decay * G
        starts.append(G)
    g["d_initial_state"] = np.array(starts).reshape(len(offsets) - 1, heads, dk, dv)
    return g


def linear_attention_step(state, q, k, v, log_decay, scale, slots=None):
    """(out, new state); entries with a negative slot give zeros."""
    state, q, k, v = (np.array(x, np.float64) for x in (state, q, k, v))
    decay = np.exp(np.asarray(log_decay, np.float64))[:, None, None]
    out = np.zeros((q.shape[0], q.shape[1], v.shape[2]))
    for b in range(q.shape[0]):
        s = b if slots is None else int(slots[b])
        if s < 0:
            continue
        state[s] = decay * state[s] + k[b][:, :, None] * v[b][:, None, :]
        out[b] = scale * np.einsum("hd,hde->he", q[b], state[s])
    return out, state
