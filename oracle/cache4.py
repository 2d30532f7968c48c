"""Oracle of the paged 4-bit key/value cache, in float64 and Python integers:
the row format, its place in a page, the page plan, and attention over cached
tokens. Follows the definitions stated in include/scfa.h."""
import numpy as np


def scale_byte(a):
    """Scale byte of a group whose largest magnitude is a: a / 7 within
    [2^-15, 9216], rounded to four significant bits, ties to even."""
    t = min(max(float(a) / 7.0, 2.0 ** -15), 9216.0)
    m, e = np.frexp(t)  # t = m 2^e, m in [0.5, 1)
    q = int(np.rint(m * 16.0))
    if q == 16:
        q, e = 8, e + 1
    return int((e + 14) * 8 + (q - 8))


def scale_value(b):
    b = np.asarray(b, np.int64)
    return (1.0 + (b & 7) / 8.0) * np.exp2((b >> 3) - 15.0)


def quantise(x):
    """Rows [..., D] -> codes -7..7 [..., D] and scale bytes [..., D / 32]."""
    x = np.asarray(x, np.float64)
    x = np.where(np.isnan(x), 0.0, x)
    g = x.reshape(*x.shape[:-1], -1, 32)
    amax = np.abs(g).max(-1)
    b = np.vectorize(scale_byte, otypes=[np.int64])(amax)
    with np.errstate(invalid="ignore"):
        c = np.clip(np.rint(g / scale_value(b)[..., None]), -7, 7)
    return c.reshape(x.shape).astype(np.int64), b


def values(x):
    """What the cache holds of rows [..., D]."""
    c, b = quantise(x)
    return c * np.repeat(scale_value(b), 32, -1)


def addresses(slot, head, ch, Hkv, D, page_size, is_v):
    """(byte, high half?, scale byte) of one channel's code in the flat cache."""
    G = D // 32
    page, at = divmod(slot, page_size)
    tile, t = divmod(at, 16)
    base = ((page * Hkv + head) * (page_size // 16) + tile) * 16 * (D + D // 16)
    g, i = divmod(ch, 32)
    if not is_v:
        j, i = divmod(i, 8)
        p = i // 2 + 4 * (i % 2)
        code = base + t * (D // 2) + (j * G + g) * 4 + p // 2
        return code, p % 2, base + 16 * D + t * G + g
    r, p = divmod(i, 4)
    u, w, b = t // 8, t // 2 % 4, t % 2
    code = base + 8 * D + (((u * 8 + r) * 4 + w) * 2 + b) * 2 * G + 2 * g + p // 2
    return code, p % 2, base + 16 * D + 16 * G + t * G + g


def row(cache, slot, head, Hkv, D, page_size, is_v):
    """float64 row of a flat uint8 cache."""
    out = np.empty(D)
    for ch in range(D):
        at, high, sc = addresses(slot, head, ch, Hkv, D, page_size, is_v)
        out[ch] = ((int(cache[at]) >> (4 * high) & 15) - 8) * scale_value(int(cache[sc]))
    return out


def plan(length, new_len, keep, free_pages, n_free, table, N, page_size, n_pages):
    """The new state and the step's tokens: a dict, or the name of the error."""
    R, max_pages = table.shape
    if min(length) < 0 or min(new_len) < 0 or sum(map(int, new_len)) > N or not 0 <= n_free <= n_pages:
        return "invalid"
    table, stack = table.copy(), list(free_pages[:n_free])
    q_start, slot, vis, out = [0], np.full(N, -1), np.zeros(N, np.int64), []
    t, short = 0, False
    for r in range(R):
        n = int(length[r])
        for _ in range(int(new_len[r])):
            if keep is None or keep[t]:
                if n // page_size >= max_pages:
                    return "invalid"
                if n % page_size == 0:
                    short = short or not stack
                    table[r, n // page_size] = stack.pop() if stack else -1
                slot[t] = table[r, n // page_size] * page_size + n % page_size
                n += 1
            vis[t] = n
            t += 1
        q_start.append(t)
        out.append(n)
    if max(-(-int(n) // page_size) for n in length) > max_pages:
        return "invalid"
    if short:
        return "no pages"
    return dict(table=table, len=np.array(out), n_free=len(stack), q_start=np.array(q_start), slot=slot, vis=vis)


def attention(q, k, v, scale):
    """One query row over the rows k, v [n, D] it sees: (o, lse)."""
    if len(k) == 0:
        return np.zeros(q.shape[-1]), -np.inf
    s = k @ q * scale
    m = s.max()
    p = np.exp(s - m)
    return (p @ v) / p.sum(), m + np.log(p.sum())
