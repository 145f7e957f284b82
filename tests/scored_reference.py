"""Attention with modified scores in 64 bits (torch, any device), straight from
the definition, and the bound on a correctly computed 16-bit result."""
import torch

BS = 16
TINY = {torch.float16: 2.0 ** -25, torch.bfloat16: 2.0 ** -134}


def attention(q, k_cache, v_cache, tables, lens, chunks, scale, softcap=0.0, slopes=None, window=0,
              starts=None, prefixes=None, num_blocks=None):
    """q [rows, Hq, D]; tables, lens, chunks, starts, prefixes: host lists.  A
    table entry outside the pool hides its block.  Returns (out, tol), float64.

    tol, by arithmetic.  With e = eps / 2 the relative error of one rounding to
    the 16-bit type, the stored weights 2^(z - m) are off by e, their sum is
    not, so sum w |V| e; the result's rounding is e |out|.  A score's fp32 error
    d shifts weights by at most 2 d relative: the dot product's D / 16 partial
    accumulations lose at most 2^-22 of sum |q k| each (2^-19 in all), and the
    cap, bias, scaling and exponent round to 2^-21 of their largest operand (the
    cap itself only where some score of the sequence comes near it: elsewhere
    tanh is taken to a relative error).
    exp2 and the running sums add 2^-18.  fp16 weights below 2^-14 are off by up
    to 2^-25 of the largest one: 2^-25 max(w) sum |V|.
    """
    dev, dt = q.device, q.dtype
    f64 = torch.float64
    e = torch.finfo(dt).eps / 2
    Hq, D = q.shape[1:]
    NB, _, Hkv, _ = k_cache.shape
    NB = num_blocks or NB
    g = Hq // Hkv
    out = torch.zeros(q.shape, dtype=f64, device=dev)
    tol = torch.full(q.shape, TINY[dt], dtype=f64, device=dev)
    row = 0
    for s, n in enumerate(lens):
        c = chunks[s] if chunks is not None else 1
        rows, row = slice(row, row + c), row + c
        if n <= 0 or c == 0:
            continue
        ids = torch.tensor(list(tables[s][:(n + BS - 1) // BS]), dtype=torch.long, device=dev)
        there = ((ids >= 0) & (ids < NB)).repeat_interleave(BS)[:n]
        ids = torch.where((ids >= 0) & (ids < NB), ids, torch.zeros_like(ids))
        t = torch.arange(n, device=dev)
        p = torch.arange(n - c, n, device=dev)[:, None]
        start = max(starts[s], 0) if starts is not None else 0
        prefix = min(max(prefixes[s], 0), n) if prefixes is not None else 0
        seen = (t >= start) & ((t <= p) | (t < prefix)) & there
        if window:
            seen &= t > p - window
        any_row = seen.any(dim=0)                        # keys some row sees
        first = int(any_row.nonzero()[0]) if any_row.any() else n
        # gather once, from the first key seen
        K = k_cache[ids[first // BS:]].reshape(-1, Hkv, D)[first % BS:first % BS + n - first].to(f64)
        V = v_cache[ids[first // BS:]].reshape(-1, Hkv, D)[first % BS:first % BS + n - first].to(f64)
        seen, t = seen[:, first:], t[first:]
        if t.numel() == 0:
            continue
        near_cap = 0.0
        for h in range(Hq if softcap else 0):
            Kh = torch.where(any_row[first:, None], K[:, h // g], torch.zeros((), dtype=f64, device=dev))
            z = (scale * (q[rows, h].to(f64) @ Kh.T)).abs()
            if bool((torch.where(torch.isnan(z), torch.full_like(z, float("inf")), z)
                     > softcap / 5).any()):
                near_cap = softcap
                break
        for h in range(Hq):
            qh = q[rows, h].to(f64)
            Kh = torch.where(any_row[first:, None], K[:, h // g], torch.zeros((), dtype=f64, device=dev))
            Vh = V[:, h // g]
            z = scale * (qh @ Kh.T)
            size = abs(scale) * (qh.abs() @ Kh.abs().T)
            if softcap:
                z = softcap * torch.tanh(z / softcap)
            big = z.abs()
            if slopes is not None:
                away = (p - t).abs().to(f64) * float(slopes[h])
                z = z - away
                big = big + away.abs()
            z = torch.where(seen, z, torch.full_like(z, -float("inf")))
            some = seen.any(dim=1, keepdim=True)
            w = torch.where(some, torch.softmax(torch.where(some, z, torch.zeros_like(z)), dim=1),
                            torch.zeros_like(z))
            w = torch.where(seen, w, torch.zeros_like(w))
            # rows of V that a query does not see never meet its weights
            def mix(weights, values):
                clean = torch.where(torch.isfinite(values), values, torch.zeros_like(values))
                r = weights @ clean
                for j in torch.nonzero(~torch.isfinite(values).all(dim=1)).flatten().tolist():
                    hit = seen[:, j]
                    r[hit] += weights[hit, j, None] * (values[j] - clean[j])[None]
                return r
            o = mix(w, Vh)
            a = mix(w, Vh.abs())
            d = 2.0 ** -19 * torch.where(seen, size, torch.zeros_like(size)).amax(1, keepdim=True)
            d = d + 2.0 ** -21 * (torch.where(seen, big, torch.zeros_like(big)).amax(1, keepdim=True)
                                  + near_cap)
            small = 2.0 ** -25 * w.amax(1, keepdim=True) * (
                seen.to(f64) @ torch.where(torch.isfinite(Vh), Vh.abs(), torch.zeros_like(Vh))
            ) if dt == torch.float16 else 0.0
            out[rows, h] = o
            tol[rows, h] = a * (e + 2 * d + 2.0 ** -18) + e * o.abs() + small + TINY[dt]
    return out, tol


def assert_close(got, out, tol, what=""):
    got = got.to(torch.float64)
    nan = torch.isnan(out)
    assert torch.equal(torch.isnan(got), nan), f"{what}: NaN pattern differs"
    inf = torch.isinf(out)
    assert torch.equal(got[inf], out[inf]), f"{what}: infinities differ"
    ok = ~nan & ~inf
    ratio = ((got - out).abs() / tol)[ok]
    assert torch.isfinite(got[ok]).all(), f"{what}: non-finite output"
    worst = float(ratio.max()) if ratio.numel() else 0.0
    assert worst <= 1.0, f"{what}: {worst:.3f} of the bound"
    return worst
