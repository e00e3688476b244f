"""The operators around the MoE layer from their definitions, in 64 bits on the host (test side only)."""
import numpy as np
import torch


def quantize_rows(v32):
    """Codes and fp32 scales of rows of fp32 values: scale = fp32(amax / 127), codes rint(fp32(v / scale))."""
    v = v32.astype(np.float32)
    amax = np.abs(v).max(axis=1, keepdims=True)
    scale = (amax / np.float32(127.0)).astype(np.float32)
    safe = np.where(scale > 0, scale, np.float32(1.0))
    q = np.clip(np.rint((v / safe).astype(np.float32)), -127, 127)
    return np.where(scale > 0, q, 0.0).astype(np.int8), scale[:, 0]


def linear(xq, sx, wq, sw, bias=None):
    """(y, |acc sx sw|) in fp64."""
    acc = (torch.from_numpy(xq.astype(np.float64)) @ torch.from_numpy(wq.astype(np.float64)).T).numpy()
    p = acc * sx.astype(np.float64)[:, None] * sw.astype(np.float64)[None, :]
    return p + (0.0 if bias is None else bias.astype(np.float64)[None, :]), np.abs(p)


def rms(v, eps):
    return np.sqrt((v * v).mean(axis=1, keepdims=True) + eps)


def sample(logits, u, temperature=None, top_k=None, top_p=None, min_p=None, allowed=None):
    """Token and probability per row; allowed: boolean [rows][vocab]."""
    rows, vocab = logits.shape
    token, prob = np.full(rows, -1, np.int32), np.zeros(rows)
    for t in range(rows):
        l = logits[t].astype(np.float64)
        ok = ~np.isnan(l) & (l != -np.inf)
        if allowed is not None:
            ok &= allowed[t]
        ids = np.flatnonzero(ok)
        if ids.size == 0:
            continue
        ids = ids[np.argsort(-l[ids], kind="stable")]
        temp = 1.0 if temperature is None else float(temperature[t])
        if not temp > 0:
            token[t], prob[t] = ids[0], 1.0
            continue
        if top_k is not None and top_k[t] > 0:
            ids = ids[:top_k[t]]
        m = l[ids[0]]
        with np.errstate(invalid="ignore"):
            e = np.where(l[ids] == m, 1.0, np.exp((l[ids] - m) / temp))
        n = ids.size
        if top_p is not None and top_p[t] < 1:
            before = np.concatenate([[0.0], np.cumsum(e)[:-1]])
            n = max(1, int((before < float(top_p[t]) * e.sum()).sum()))
        if min_p is not None and min_p[t] > 0:
            n = min(n, int((e >= min(float(min_p[t]), 1.0)).sum()))
        by = np.argsort(ids[:n], kind="stable")
        ids, e = ids[:n][by], e[:n][by]
        cum = np.cumsum(e)
        at = min(n - 1, int((cum <= float(u[t]) * cum[-1]).sum()))
        token[t], prob[t] = ids[at], e[at] / cum[-1]
    return token, prob


def pack_bits(allowed):
    """[rows][vocab] booleans as [rows][ceil(vocab / 32)] int32 words, bit i of word j for token 32 j + i."""
    rows, vocab = allowed.shape
    pad = np.zeros((rows, (vocab + 31) // 32 * 32), bool)
    pad[:, :vocab] = allowed
    return np.packbits(pad, axis=1, bitorder="little").view(np.int32)
