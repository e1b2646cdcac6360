"""fp64 reference of linear attention with one decay per head, token by token
(numpy; no chunks, no code of the HIP path), and of beam search's selection.

  S_t = lam S_{t-1} + k_t v_t^T,  o_t = scale S_t^T q_t,  lam = exp(g_h)
  R_t = dL/dS_t = lam R_{t+1} + scale q_t do_t^T (the last one plus ds_final)
  dq_t = scale S_t do_t, dk_t = R_t v_t, dv_t = R_t^T k_t, ds0 = lam R_0,
  dg = sum_t <R_t, lam S_{t-1}>
"""
from __future__ import annotations

import numpy as np


def _f64(*xs):
    return [None if x is None else np.asarray(x, dtype=np.float64) for x in xs]


def _shared(x, H):
    """[T, Hk, D] -> [T, H, D]: query head h reads head h // (H / Hk)."""
    return np.repeat(x, H // x.shape[1], axis=1)


def forward(q, k, v, g, s0=None, scale=1.0):
    """One sequence: q [T,H,Dk], k [T,Hk,Dk], v [T,Hk,Dv], g [H], s0 [H,Dk,Dv].
    Returns (o [T,H,Dv], the states S_{-1} .. S_{T-1} [T+1,H,Dk,Dv])."""
    q, k, v, g, s0 = _f64(q, k, v, g, s0)
    T, H, Dk = q.shape
    k, v = _shared(k, H), _shared(v, H)
    lam = np.exp(g)[:, None, None]
    S = np.zeros((H, Dk, v.shape[2])) if s0 is None else s0
    states, o = [S], np.zeros((T, H, v.shape[2]))
    for t in range(T):
        S = lam * S + k[t][:, :, None] * v[t][:, None, :]
        o[t] = scale * np.einsum("hkv,hk->hv", S, q[t])
        states.append(S)
    return o, np.stack(states)


def backward(q, k, v, g, d_o, s0=None, ds_final=None, scale=1.0):
    """Gradients of one sequence, as a dict (dk, dv summed over shared heads)."""
    q, k, v, g, d_o, ds_final = _f64(q, k, v, g, d_o, ds_final)
    T, H, Dk = q.shape
    Hk = k.shape[1]
    _, S = forward(q, k, v, g, s0, scale)
    ke, ve = _shared(k, H), _shared(v, H)
    lam = np.exp(g)[:, None, None]
    R = np.zeros_like(S[0]) if ds_final is None else ds_final
    dq, dk, dv, dg = np.zeros(q.shape), np.zeros(ke.shape), np.zeros(ve.shape), np.zeros(H)
    for t in reversed(range(T)):
        R = R + scale * q[t][:, :, None] * d_o[t][:, None, :]
        dq[t] = scale * np.einsum("hkv,hv->hk", S[t + 1], d_o[t])
        dk[t] = np.einsum("hkv,hv->hk", R, ve[t])
        dv[t] = np.einsum("hkv,hk->hv", R, ke[t])
        dg += (R * lam * S[t]).sum((1, 2))
        R = lam * R
    group = lambda x: x.reshape(T, Hk, H // Hk, x.shape[2]).sum(2)  # noqa: E731
    return {"dq": dq, "dk": group(dk), "dv": group(dv), "dg": dg, "ds0": R}


def select(logits, scores, done=None, eos=-1, pad=0):
    """beam_select of one request: logits [K,V], scores [K], done [K] or None."""
    logits, scores = _f64(logits, scores)
    K, V = logits.shape
    cand = np.full((K, V), -np.inf)
    with np.errstate(all="ignore"):
        for k in range(K):
            if done is not None and done[k]:
                cand[k, pad] = scores[k]
            else:
                m = logits[k].max()
                cand[k] = scores[k] + (logits[k] - (m + np.log(np.exp(logits[k] - m).sum())))
    cand[~np.isfinite(cand)] = -np.inf
    flat = np.argsort(-cand.reshape(-1), kind="stable")[:K]
    tokens, parents = flat % V, flat // V
    ended = (tokens == eos) | (np.zeros(K, bool) if done is None else np.asarray(done, bool)[parents])
    return cand.reshape(-1)[flat], tokens, parents, ended
