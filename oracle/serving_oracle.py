"""fp64 oracle of the operators around the prefill path: rotary positions,
paged append and paged attention (plain NumPy, no code shared with the CUDA
path; test infrastructure only)."""

import math

import numpy as np

from oracle.dhsa_oracle import as_f64


def rope_frequencies(rotary_dim, base, scaling=None):
    """(frequencies in radians a position, factor on cos and sin), pair by pair."""
    out, factor = [], 1.0
    for i in range(rotary_dim // 2):
        f = math.pow(base, -2.0 * i / rotary_dim)
        if scaling is None:
            pass
        elif scaling.kind == "linear":
            f /= scaling.factor
        elif scaling.kind == "llama3":
            wave = 2 * math.pi / f
            longest = scaling.original_len / scaling.low_freq_factor
            shortest = scaling.original_len / scaling.high_freq_factor
            if wave > longest:
                f /= scaling.factor
            elif wave >= shortest:
                x = (scaling.original_len / wave - scaling.low_freq_factor) / (
                    scaling.high_freq_factor - scaling.low_freq_factor)
                f = (1 - x) * f / scaling.factor + x * f
        elif scaling.kind == "yarn":
            def pair(turns):
                return rotary_dim * math.log(scaling.original_len / (2 * math.pi * turns)) / (2 * math.log(base))
            lo = max(math.floor(pair(scaling.beta_fast)), 0)
            hi = min(math.ceil(pair(scaling.beta_slow)), rotary_dim - 1)
            w = min(max((i - lo) / ((hi - lo) or 0.001), 0.0), 1.0)
            f = w * f / scaling.factor + (1 - w) * f
            factor = 0.1 * math.log(scaling.factor) + 1.0
        else:
            raise ValueError(scaling.kind)
        out.append(f)
    return np.array(out), factor


def rope(x, positions, freqs, factor=1.0, interleaved=False):
    """x [T, H, d] rotated at integer positions [T]."""
    y = as_f64(x).copy()
    n = len(freqs)
    angle = np.asarray(positions, dtype=np.float64)[:, None, None] * np.asarray(freqs)
    first = slice(0, 2 * n, 2) if interleaved else slice(0, n)
    second = slice(1, 2 * n, 2) if interleaved else slice(n, 2 * n)
    turned = (y[..., first] + 1j * y[..., second]) * (factor * np.exp(1j * angle))
    y[..., first], y[..., second] = turned.real, turned.imag
    return y


def append(k_pages, v_pages, k, v, cu_q, kv_lens, table):
    """Pages (fp64 copies) with the new (already rotated) k and v stored."""
    kp, vp = as_f64(k_pages).copy(), as_f64(v_pages).copy()
    page = kp.shape[2]
    for b in range(len(cu_q) - 1):
        n = cu_q[b + 1] - cu_q[b]
        for j in range(n):
            s = int(kv_lens[b]) - n + j
            if s < 0:
                continue
            kp[table[b][s // page], :, s % page] = as_f64(k[cu_q[b] + j])
            vp[table[b][s // page], :, s % page] = as_f64(v[cu_q[b] + j])
    return kp, vp


def paged_attention(q, k_pages, v_pages, cu_q, kv_lens, table, group_ptr=None, prefix_lens=None, scale=None):
    """(out [T, Hq, d], lse [T, Hq]) token by token, over the keys it sees: the
    first prefix_lens[g] from the table row of its group's first sequence."""
    q, kp, vp = as_f64(q), as_f64(k_pages), as_f64(v_pages)
    T, hq, d = cu_q[-1], q.shape[1], q.shape[2]
    hkv, page = kp.shape[1], kp.shape[2]
    r = hq // hkv
    scale = 1 / math.sqrt(d) if scale is None else scale
    out, lse = np.zeros((T, hq, d)), np.full((T, hq), -np.inf)
    for b in range(len(cu_q) - 1):
        n, held = cu_q[b + 1] - cu_q[b], int(kv_lens[b])
        shared, first = 0, b
        if group_ptr is not None:
            g = int(np.searchsorted(group_ptr, b, side="right") - 1)
            shared, first = int(prefix_lens[g]), int(group_ptr[g])
        where = [(table[first if s < shared else b][s // page], s % page) for s in range(held)]
        keys = np.array([kp[p, :, x] for p, x in where]).reshape(held, hkv, d)
        vals = np.array([vp[p, :, x] for p, x in where]).reshape(held, hkv, d)
        for j in range(n):
            seen = held - n + j + 1
            if seen <= 0:
                continue
            t = cu_q[b] + j
            x = np.einsum("grd,sgd->grs", q[t].reshape(hkv, r, d), keys[:seen]) * scale
            top = x.max(-1, keepdims=True)
            e = np.exp(x - top)
            out[t] = (np.einsum("grs,sgd->grd", e, vals[:seen]) / e.sum(-1, keepdims=True)).reshape(hq, d)
            lse[t] = (top[..., 0] + np.log(e.sum(-1))).reshape(hq)
    return out, lse
