"""Plain 64-bit statements of the mixture-of-experts token operators and of
the low-rank adapters, for the tests to compare with (numpy, token by token;
nothing is shared with the library)."""
import numpy as np

MASK_AT = -3.3895313892515355e38  # bf16's lowest finite value


def route(logits, top_k, score="softmax", bias=None, groups=1, top_groups=1, group_top=1,
          renormalize=True, scale=1.0):
    """(ids int64 [M, k], weights float64 [M, k]) of float logits [M, E]."""
    logits = np.asarray(logits, np.float64)
    M, E = logits.shape
    ids = np.full((M, top_k), -1, np.int64)
    weights = np.zeros((M, top_k))
    size = E // groups
    for m in range(M):
        l = logits[m]
        ok = np.array([not np.isnan(v) and v > MASK_AT for v in l])
        if not ok.any():
            continue
        p = np.zeros(E)
        if score == "sigmoid":
            with np.errstate(over="ignore"):
                p[ok] = 1.0 / (1.0 + np.exp(-l[ok]))
        elif np.isposinf(l[ok]).any():
            p[ok] = np.isposinf(l[ok]) / np.isposinf(l[ok]).sum()
        else:
            e = np.exp(l[ok] - l[ok].max())
            p[ok] = e / e.sum()
        key = l if bias is None else p + np.asarray(bias, np.float64)
        open_ = ok.copy()
        if groups > 1:
            val = []
            for g in range(groups):
                at = [e for e in range(g * size, (g + 1) * size) if ok[e]]
                src = p if (bias is None and group_top == 2) else key
                best = sorted((src[e] for e in at), reverse=True)[:group_top]
                val.append(sum(best) if best else -np.inf)
            used = sorted(range(groups), key=lambda g: (-val[g], g))[:top_groups]
            for g in range(groups):
                if g not in used:
                    open_[g * size:(g + 1) * size] = False
        at = sorted((e for e in range(E) if open_[e]), key=lambda e: (-key[e], e))[:top_k]
        if not at:
            continue
        w = p[at]
        if renormalize:
            if score == "softmax":
                x = l[at]
                w = np.isposinf(x).astype(float) if np.isposinf(x).any() else np.exp(x - x.max())
            else:  # by logarithms, as small scores keep their proportions
                x = -np.logaddexp(0.0, -l[at])
                w = np.exp(x - x.max())
            w = w / w.sum()
        ids[m, :len(at)] = at
        weights[m, :len(at)] = w * scale
    return ids, weights


def places(ids, groups):
    """(offsets, rows, pos) of ids [M, k]: the stable order by id."""
    flat = np.asarray(ids).reshape(-1)
    rows = [i for g in range(groups) for i in np.nonzero(flat == g)[0]]
    pos = np.full(flat.size, -1, np.int64)
    for at, i in enumerate(rows):
        pos[i] = at
    offsets = np.concatenate([[0], np.cumsum([(flat == g).sum() for g in range(groups)])])
    return offsets, np.array(rows, np.int64), pos.reshape(np.shape(ids))


def combine(Y, pos, weights):
    """(out, the sum of the terms' magnitudes), float64."""
    M, k = pos.shape
    out = np.zeros((M, Y.shape[1]))
    mag = np.zeros_like(out)
    for m in range(M):
        for j in range(k):
            if 0 <= pos[m, j] < Y.shape[0]:
                t = np.float64(weights[m, j]) * Y[pos[m, j]].astype(np.float64)
                out[m] += t
                mag[m] += np.abs(t)
    return out, mag


def lora(X, Y, A, B, ids, scale):
    """(Y + scale B A x, error bound of an fp32 evaluation that takes fp32
    values in two bf16 terms), float64 arrays in."""
    K, r = A.shape[2], A.shape[1]
    out = Y.copy()
    tol = np.zeros_like(Y)
    for a in range(A.shape[0]):
        at = np.nonzero(ids == a)[0]
        if not len(at):
            continue
        s = 1.0 if scale is None else scale[a]
        t = X[at] @ A[a].T
        out[at] += s * (t @ B[a].T)
        # two bf16 terms leave 2^-16 of a value; a product of sixteen terms
        # into an fp32 sum is off by at most 2^-22 of the terms so far, and
        # there are K / 16 (r / 16) such steps for each of the two terms
        e1 = (2.0 ** -16 + (K / 8 + 32) * 2.0 ** -22) * (np.abs(X[at]) @ np.abs(A[a]).T)
        e2 = (2.0 ** -16 + (r / 8 + 32) * 2.0 ** -22) * (np.abs(t) @ np.abs(B[a]).T)
        tol[at] += abs(s) * (e1 @ np.abs(B[a]).T + e2) + 2.0 ** -22 * np.abs(Y[at])
    return out, tol
