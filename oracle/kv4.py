"""fp64 definition of the 4-bit paged key-value cache: number formats, layout, page plan, attention (numpy)."""
import numpy as np

E2M1 = np.array([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0])
_b = np.arange(256)
_e, _m = (_b >> 3) & 15, _b & 7
E4M3 = np.where(_e > 0, (1 + _m / 8) * 2.0 ** (_e - 7), _m * 2.0 ** -9) * np.where(_b > 127, -1.0, 1.0)
E4M3[[0x7F, 0xFF]] = np.nan


def _nearest(x, there):
    """Index of the value of the ascending list `there` nearest to x >= 0, ties to the even index, saturating."""
    hi = np.clip(np.searchsorted(there, x), 1, len(there) - 1)
    lo = hi - 1
    below, above = x - there[lo], there[hi] - x
    return np.where((above < below) | ((above == below) & (hi % 2 == 0)), hi, lo)


def quantize(x, factor):
    """x [..., d] -> codes [..., d] (0 .. 15), scale bytes [..., d / 16], values [..., d]."""
    x = np.asarray(x, np.float64)
    y = x.reshape(*x.shape[:-1], -1, 16) / factor
    bad = np.isnan(y).any(-1, keepdims=True)
    y = np.where(bad, 0.0, y)
    top = np.minimum(np.abs(y).max(-1, keepdims=True) / 6.0, 1e9)
    scale = _nearest(top, E4M3[:0x7F])
    s = E4M3[scale]
    u = np.divide(np.minimum(np.abs(y), 1e30), s, out=np.zeros_like(y), where=s > 0)
    mag = _nearest(np.minimum(u, 6.0), E2M1)
    code = np.where(s > 0, mag + 8 * np.signbit(y), 0)
    values = np.where(bad, np.nan, E2M1[code & 7] * np.where(code > 7, -1.0, 1.0) * s * factor)
    scale = np.where(bad, 0x7F, scale)
    return code.reshape(x.shape).astype(np.uint8), scale[..., 0].astype(np.uint8), values.reshape(x.shape)


def places(key, col, d):
    """(byte, shift) of a K code, (byte, shift) of a V code, byte of the K scale, byte of the V scale, within a tile."""
    t, c, p = key // 8, key % 8 // 2, key % 2
    grp, g = col // 16, col // (d // 8)
    kb = key * (d // 2) + col // 2
    vb = 8 * d + (((t * 8 + g) * 4 + c) * 2 + p) * (d // 16) + (col % (d // 8)) // 2
    ks = 16 * d + ((key % 8) * (d // 16) + grp) * 2 + t
    vs = 17 * d + (grp * 4 + c) * 4 + t * 2 + p
    return kb, vb, 4 * (col % 2), ks, vs


def store(cache, slot, k, v, k_factor, v_factor):
    """Write one token's k, v [H_kv, d] to a slot of cache [pages, H_kv, P / 16, 18 d] (uint8, in place)."""
    d = k.shape[-1]
    page_size = cache.shape[2] * 16
    tile = cache[slot // page_size, :, slot % page_size // 16]
    key = slot % 16
    col = np.arange(d)
    kb, vb, sh, ks, vs = places(key, col, d)
    for x, at, sc, f in ((k, kb, ks, k_factor), (v, vb, vs, v_factor)):
        code, scale, _ = quantize(x, f)
        for h in range(k.shape[0]):
            tile[h, at[::2]] = code[h, ::2] | code[h, 1::2] << 4
            tile[h, sc[::16]] = scale[h]


def read(cache, table_row, n, k_factor, v_factor):
    """K, V [H_kv, n, d] of one request."""
    d = cache.shape[3] // 18
    page_size = cache.shape[2] * 16
    pos = np.arange(n)
    tiles = cache[np.asarray(table_row)[pos // page_size], :, pos % page_size // 16]  # [n, H_kv, 18 d]
    key, col = pos[:, None] % 16, np.arange(d)[None]
    kb, vb, sh, ks, vs = places(key, col, d)
    take = lambda at: np.take_along_axis(tiles, np.broadcast_to(at, (n, d))[:, None], 2)  # noqa: E731
    code = lambda at: (take(at) >> sh[:, None] if np.ndim(sh) > 1 else take(at) >> sh) & 15  # noqa: E731
    val = lambda c: E2M1[c & 7] * np.where(c > 7, -1.0, 1.0)  # noqa: E731
    k = val(code(kb)) * E4M3[take(ks)] * k_factor
    v = val(code(vb)) * E4M3[take(vs)] * v_factor
    return k.transpose(1, 0, 2), v.transpose(1, 0, 2)


def plan(cached, new, free, table, page_size, max_tokens):
    """The page plan: (table, lens, cu_new, cu_total, slots, positions, pages_needed)."""
    table = np.array(table)
    slots, positions, cu_new, cu_total, lens, taken = [], [], [0], [0], [], 0
    for b, (c, n) in enumerate(zip(cached, new)):
        if c < 0 or n < 0 or c + n > table.shape[1] * page_size:
            c = n = 0
        for i in range(-(-c // page_size), -(-(c + n) // page_size)):
            table[b, i] = free[taken] if taken < len(free) else -1
            taken += 1
        for pos in range(c, c + n):
            page = table[b, pos // page_size]
            slots.append(int(page) * page_size + pos % page_size if page >= 0 else -1)
            positions.append(pos)
        lens.append(c + n)
        cu_new.append(cu_new[-1] + n)
        cu_total.append(cu_total[-1] + c + n)
    pad = max_tokens - len(slots)
    slots, positions = (slots + [-1] * pad)[:max_tokens], (positions + [0] * pad)[:max_tokens]
    return table, lens, cu_new, cu_total, slots, positions, taken


def attention(q, k, v, scale, causal):
    """q [Lq, H, d], k, v [H_kv, Lk, d] -> o [Lq, H, d], lse [H, Lq], and for error bounds sum p |v| [Lq, H, d] and
    the largest scale * sum |q| |k| of a row [H, Lq].  Keys a query does not see have no influence."""
    lq, H, d = q.shape
    hkv, lk = k.shape[:2]
    G = H // hkv
    o, mass = np.zeros((lq, H, d)), np.zeros((lq, H, d))
    lse, size = np.full((H, lq), -np.inf), np.zeros((H, lq))
    for i in range(lq):
        see = max(0, lk - lq + i + 1) if causal else lk
        if see == 0:
            continue
        for h in range(hkv):
            x = np.asarray(q[i, h * G:(h + 1) * G], np.float64)
            kk, vv = k[h, :see], v[h, :see]
            s = scale * (x @ kk.T)
            m = s.max(-1, keepdims=True)
            e = np.exp(s - m)
            z = e.sum(-1, keepdims=True)
            o[i, h * G:(h + 1) * G] = (e / z) @ vv
            mass[i, h * G:(h + 1) * G] = (e / z) @ np.abs(vv)
            lse[h * G:(h + 1) * G, i] = (m + np.log(z))[:, 0]
            size[h * G:(h + 1) * G, i] = scale * (np.abs(x) @ np.abs(kk).T).max(-1)
    return o, lse, mass, size
