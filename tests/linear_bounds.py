"""How far the gradient of linear attention's decays may be off (shared by its tests on the GPU and on the CPU).

dlog_decay_t is the sum of what passes token t: an addend is a product of a query, a key, two rows of do and v and the decays between
them, in which t's own always is.  In fp32 each passes at most n = 2 (K + V) + L / 16 + 200 roundings of 2^-24 (both
contractions, the chunk's sums, one product and sum a chunk), and e^x is off by 2^-24 |x| for the exponents' own
rounding.  With m(g) the sum of the addends' magnitudes, the sum of |x| times them is at most (m((1 - h) g) - m(g)) / h
for every h > 0, e^-(1-h)x - e^-x being at least h x e^-x.

What passes a whole chunk, Z, follows from the chunk behind it within spans of 8 chunks, so it has the 2^-24 of what
that is formed of: the x and y on the way to the span's end, or to a chunk in which a token starts anew or whose decay is below 2^-149,
and <S, R> there.  Not in spans with a chunk that has a token below 2^-6 and is neither: there Z has only its own.

These are worst cases.  Roundings are as often up as down: an addend's are off by 2^-25 n^1/2 in the mean square, and the 2 * 8 *
64 rows of x and y that Z is formed of by 32 times that of one, together by less than NORM = 32 * 25 * 2^-25 of a row, while
the gradient of a head sums at least one.  So a head's gradients are off by NORM in relative norm at most, unless they vanish."""
import numpy as np

from oracle import linear as orc

SPAN = 8
NORM = 32 * 25 * 2.0 ** -25


def chunk_of(io, K, V):
    return 32 if io == "f32" and max(K, V) > 128 else 64


def absolute(i):
    return {k: (np.abs(v) if k in ("q", "k", "v", "do", "S0", "dlast") and v is not None else v) for k, v in i.items()}


def parts(i, size, io, S0=True, dlast=True, chunk=None):
    return orc.linear_decay_parts(i["q"], i["k"], i["v"], i["g"], i["do"], i["scale"], i["S0"] if S0 else None,
                                  i["dlast"] if dlast else None, chunk or chunk_of(io, size[4], size[5]))


def marked(p, n, S0, dlast):
    """[B, chunks, H]: whether a chunk's span has one that is to have its own product."""
    own = (p["least"] < -6.0) & ~p["starts"] & (p["log2"] > -149.0)
    if not S0:
        own[:, 0] = False
    if not dlast:
        own[:, -1] = False
    out = np.zeros_like(own)
    for s in range(0, n, SPAN):
        out[:, s:s + SPAN] = own[:, s:s + SPAN].any(1, keepdims=True)
    return out


def decay_bound(i, size, io, S0=True, dlast=True):
    """(dlog_decay [B, L, H], its bound)."""
    B, L, H, Hk, K, V = size
    chunk = chunk_of(io, K, V)
    n, u, h = 2 * (K + V) + L / 16 + 200, 2.0 ** -24, 0.05
    ref = parts(i, size, io, S0, dlast)
    a = absolute(i)
    mag = parts(a, size, io, S0, dlast)
    with np.errstate(invalid="ignore"):
        slower = parts(dict(a, g=np.asarray(a["g"], np.float64) * (1 - h)), size, io, S0, dlast)
    bound = n * u * mag["dlog_decay"] + 2 * u * np.abs(slower["dlog_decay"] - mag["dlog_decay"]) / h
    chunks = ref["through"].shape[1]
    cut = ref["starts"] | (ref["log2"] < -149.0)
    if not S0:
        cut[:, 0] = True
    if not dlast:
        cut[:, -1] = True
    own = marked(ref, chunks, S0, dlast)
    on_way = np.zeros((B, H))
    for c in range(chunks - 1, -1, -1):
        r = slice(c * chunk, min(L, (c + 1) * chunk))
        x, y = mag["x"][:, r].sum(1), mag["y"][:, r].sum(1)
        if c % SPAN == SPAN - 1 or c == chunks - 1:
            on_way = mag["beside"][:, c]
        bound[:, r] += np.where(cut[:, c] | own[:, c], 0.0, n * u * (on_way + y))[:, None]
        on_way = np.where(cut[:, c], x, on_way + y + x)
    start = np.broadcast_to(np.asarray(i["g"], np.float64), (B, L, H)) * np.log2(np.e) < -150.0
    return ref["dlog_decay"], np.where(start, 0.0, bound)


def norms(d, ref):
    """Relative norm of d over the tokens of each (batch row, head)."""
    return np.sqrt((d ** 2).sum(1) / np.maximum((ref ** 2).sum(1), 1e-280))
