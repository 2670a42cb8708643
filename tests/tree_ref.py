"""The draft-tree operators in float64, written from their definitions
(include/hogwild.h), and the inputs of their tests."""
from __future__ import annotations

import numpy as np
import torch


def rotate(x, pos, theta):
    """x [..., D] float64 rotated at pos (broadcast over the leading dims)."""
    half = x.shape[-1] // 2
    w = theta ** (-np.arange(half) / half)
    ang = np.asarray(pos, np.float64)[..., None] * w
    c, s = np.cos(ang), np.sin(ang)
    a, b = x[..., :half], x[..., half:]
    return np.concatenate([a * c - b * s, b * c + a * s], -1)


def depths(parent, n):
    d = []
    for i in range(n):
        d.append(0 if parent[i] < 0 else d[parent[i]] + 1)
    return np.asarray(d, np.int64)


def ancestors(parent, n):
    m = np.zeros((n, n), bool)
    for i in range(n):
        if parent[i] >= 0:
            m[i] = m[parent[i]]
        m[i, i] = True
    return m


def random_parents(rng, rows, T, kind, n_nodes):
    out = np.full((rows, T), -1, np.int32)
    for r in range(rows):
        for i in range(1, int(n_nodes[r])):
            out[r, i] = i - 1 if kind == "chain" else int(rng.integers(-1 if kind == "forest" else 0, i))
    return out


def attend(*, q, k, v, block_start, block_len, views, offsets, q_pos, tree_block, tree_start, n_nodes,
           parent, heads, scale, theta):
    """out, lse, spread: q [R][T][Hq][D]; k, v [Hkv][cap][D] with the trees'
    tokens in place (all float64); heads[hq] its kv head.  spread[r][i][hq]:
    sum_j p_j |v_j| [D] and the largest sum_d |q~_d k_d| scale, for bounds."""
    R, T, Hq, D = q.shape
    out = np.zeros(q.shape)
    lse = np.full((R, T, Hq), -np.inf)
    absv = np.zeros(q.shape)
    reach = np.zeros((R, T, Hq))
    for r in range(R):
        n = int(n_nodes[r])
        if n == 0:
            continue
        dep, anc = depths(parent[r], n), ancestors(parent[r], n)
        for hq in range(Hq):
            g = heads[hq]
            s_all, v_all, a_all = [], [], []
            for b, o in zip(views[r], offsets[r]):
                if b < 0 or block_len[b] <= 0:
                    continue
                kk = k[g, block_start[b]:block_start[b] + block_len[b]]
                qt = rotate(q[r, :n, hq], int(q_pos[r]) + dep - int(o), theta)
                s_all.append(qt @ kk.T * scale)
                a_all.append(np.abs(qt) @ np.abs(kk).T * scale)
                v_all.append(v[g, block_start[b]:block_start[b] + block_len[b]])
            kk = k[g, tree_start[r]:tree_start[r] + n]
            qt = rotate(q[r, :n, hq], int(block_len[tree_block[r]]) + dep, theta)
            s_all.append(np.where(anc, qt @ kk.T * scale, -np.inf))
            a_all.append(np.where(anc, np.abs(qt) @ np.abs(kk).T * scale, 0))
            v_all.append(v[g, tree_start[r]:tree_start[r] + n])
            s, vv = np.concatenate(s_all, 1), np.concatenate(v_all, 0)
            m = s.max(1, keepdims=True)
            e = np.exp(s - m)
            p = e / e.sum(1, keepdims=True)
            out[r, :n, hq] = p @ vv
            absv[r, :n, hq] = p @ np.abs(vv)
            reach[r, :n, hq] = np.concatenate(a_all, 1).max(1)
            lse[r, :n, hq] = (m + np.log(e.sum(1, keepdims=True)))[:, 0]
    return out, lse, absv, reach


def verify(n_nodes, parent, token, p, q, u_accept, u_sample):
    """path, n_path, next_token of one row, in float64, renormalising after
    every rejection as the method is usually written."""
    T, V = p.shape
    n = int(n_nodes)
    bad = n < 0 or n > T
    if not bad:
        for i in range(n):
            bad |= not -1 <= parent[i] < i or (i > 0 and not 0 <= token[i] < V)
    if bad or n == 0:
        return [-1] * T, 0, -1

    def clean(x):
        return np.clip(np.nan_to_num(x.astype(np.float64), nan=0.0, posinf=1.0, neginf=0.0), 0, 1)

    at, path = 0, [0]
    while True:
        dist, took = clean(p[at]), None
        left = 1.0  # the mass the distribution is normalised by
        for i in [i for i in range(at + 1, n) if parent[i] == at]:
            x = token[i]
            if q is None:
                if float(u_accept[i]) * left < dist[x]:
                    took = i
                    break
                left = max(0.0, left - dist[x])
                dist[x] = 0.0
            else:
                draft = clean(q[at])
                if float(u_accept[i]) * draft[x] * left < dist[x]:
                    took = i
                    break
                rest = np.maximum(dist - left * draft, 0)
                if rest.sum() > 0:
                    dist, left = rest, rest.sum()
        if took is None:
            break
        at = took
        path.append(at)
    cum = np.cumsum(dist)
    nxt = -1 if cum[-1] <= 0 else min(V - 1, int((cum <= float(u_sample) * cum[-1]).sum()))
    return path + [-1] * (T - len(path)), len(path), nxt


def to_np(t):
    return t.detach().double().cpu().numpy()


def dev(x, dtype=torch.int32):
    return torch.as_tensor(np.asarray(x)).to("cuda", dtype)
